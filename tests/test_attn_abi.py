"""The C ABI of rotate, append and attend: every declared function is exported,
and bad arguments are refused on the host, before any HIP call (no GPU needed); the
binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qmv_attn.h")


@pytest.fixture(scope="module")
def L():
    from bit_quantized_gemv_amd import ops, qmv
    if not os.path.exists(qmv.library_path()):
        from bit_quantized_gemv_amd import build
        build.build()
    return ops._load()


def test_declared_and_exported(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", src)))
    assert names == ["qmv_append", "qmv_attend", "qmv_attend_workspace", "qmv_rotate"]
    for n in names:
        assert hasattr(L, n), n


def test_status_strings():
    from bit_quantized_gemv_amd import qmv
    for i, n in enumerate(["QMV_E_HEADS", "QMV_E_CACHE"], 16):
        assert qmv.status_string(i) == n
        assert re.search(rf"\b{n}\s*=\s*{i}\b", open(HEADER).read())


# fake, aligned, far-apart addresses: the checks fail before any use
def at(i):
    return (1 << 20) + (i << 44)


ROT = dict(freqs=at(0), positions=at(1), axes=at(2), q_weight=at(3), k_weight=at(4), positions_row=7, eps=1e-6, rot=64, n_axes=2,
           interleaved=0, w_dt=2)
CACHE = dict(k=at(5), v=at(6), k_page=16 * 2 * 128, k_slot=2 * 128, k_head=128, v_page=16 * 2 * 128, v_slot=2 * 128, v_head=128,
             pages=at(7), starts=at(8), lengths=at(9), pages_row=10, n_pages=50, page_size=16, n_seqs=3, max_pages=10, heads=2,
             head_size=128, dt=2)
BAD_ROT = [(dict(freqs=0), 1), (dict(w_dt=1), 7), (dict(rot=12), 16), (dict(rot=-8), 16), (dict(rot=136), 16), (dict(n_axes=0), 16),
           (dict(n_axes=9), 16), (dict(positions_row=-1), 15), (dict(freqs=at(0) + 2), 6), (dict(positions=at(1) + 1), 6),
           (dict(q_weight=at(3) + 8), 6), (dict(k_weight=at(4) + 2), 6)]
BAD_CACHE = [*[({n: 0}, 1) for n in ("k", "v", "pages", "starts", "lengths")], (dict(k=at(5) + 8), 6), (dict(v=at(6) + 2), 6),
             (dict(pages=at(7) + 1), 6), (dict(starts=at(8) + 2), 6), (dict(lengths=at(9) + 3), 6), (dict(k_page=16 * 256 + 4), 6),
             (dict(v_head=130), 6), (dict(dt=0), 7), (dict(dt=5), 7), (dict(k_slot=-8), 15), (dict(v_page=(1 << 40) + 8), 15),
             (dict(pages_row=-1), 15), (dict(n_pages=1 << 30, k_page=1 << 40), 15), (dict(heads=0), 16), (dict(head_size=0), 16),
             (dict(head_size=12), 16), (dict(head_size=264), 16), (dict(heads=3), 16), (dict(heads=1025), 16), (dict(n_pages=0), 17),
             (dict(page_size=0), 17), (dict(page_size=65537), 17), (dict(n_seqs=0), 17), (dict(n_seqs=65536), 17), (dict(max_pages=0), 17),
             (dict(max_pages=1 << 30), 17)]


def structs(kw):
    from bit_quantized_gemv_amd import ops
    r, c = ops.Rotation(), ops.Cache()
    for s, base in ((r, ROT), (c, CACHE)):
        for n, v in base.items():
            setattr(s, n, kw.get(n, v))
    return ctypes.byref(r), ctypes.byref(c)


CALL = dict(q=at(20), kk=at(21), vv=at(22), qo=at(23), ko=at(24), T=7, hq=8, hk=2, D=128, qt=1024, qh=128, kt=256, kh=128, vt=256, vh=128,
            xdt=2, odt=2)


@pytest.mark.parametrize("kw,code", BAD_ROT + [
    *[({n: 0}, 1) for n in ("q", "kk", "qo", "ko")], (dict(positions=0), 1), (dict(q=at(20) + 8), 6), (dict(ko=at(24) + 4), 6),
    (dict(qt=1025), 6), (dict(kh=4), 6), (dict(xdt=1), 7), (dict(odt=0), 7), (dict(qo=at(20)), 9), (dict(ko=at(1)), 9), (dict(ko=at(23)), 9),
    (dict(qt=-8), 15), (dict(kt=(1 << 40) + 8), 15), (dict(hq=0), 16), (dict(hk=1025), 16), (dict(D=4), 16), (dict(D=264), 16), (dict(T=0), 17),
    (dict(T=(1 << 22) + 1), 17)])
def test_rotate_refuses(L, kw, code):
    a = {**CALL, **kw}
    r, _ = structs(kw)
    assert L.qmv_rotate(r, *[a[n] for n in ("q", "kk", "qo", "ko", "T", "hq", "hk", "D", "qt", "qh", "kt", "kh", "xdt", "odt")], None) == code


@pytest.mark.parametrize("kw,code", BAD_ROT + BAD_CACHE + [
    *[({n: 0}, 1) for n in ("q", "kk", "vv", "qo")], (dict(q=at(20) + 8), 6), (dict(vv=at(22) + 4), 6), (dict(vt=257), 6), (dict(xdt=1), 7),
    (dict(qo=at(22)), 9), (dict(qo=at(6)), 9), (dict(k=at(21)), 9), (dict(v=at(5)), 9), (dict(pages=at(6) + 64), 9), (dict(vh=-8), 15),
    (dict(k_slot=0), 15), (dict(v_page=16 * 256 - 8), 15), (dict(k_head=64), 15), (dict(hq=0), 16), (dict(hq=7), 16), (dict(T=0), 17),
    (dict(T=(1 << 22) + 1), 17)])
def test_append_refuses(L, kw, code):
    a = {**CALL, **kw}
    r, c = structs(kw)
    assert L.qmv_append(r, c, *[a[n] for n in ("q", "kk", "vv", "qo", "T", "hq", "qt", "qh", "kt", "kh", "vt", "vh", "xdt")], None) == code


ATTEND = dict(q=at(20), out=at(23), ws=at(24), nws=1 << 40, T=7, hq=8, qt=1024, qh=128, mn=7, ml=160, window=0, sinks=0, scale=0.1, odt=2)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    *[({n: 0}, 1) for n in ("q", "out", "ws")], (dict(q=at(20) + 8), 6), (dict(out=at(23) + 2), 6), (dict(ws=at(24) + 4), 6), (dict(qt=1025), 6),
    (dict(odt=1), 7), (dict(out=at(20)), 9), (dict(out=at(5) + 16), 9), (dict(out=at(8)), 9), (dict(qh=-8), 15), (dict(hq=0), 16),
    (dict(hq=9), 16), (dict(T=0), 17), (dict(T=(1 << 22) + 1), 17), (dict(mn=0), 17), (dict(ml=-1), 17), (dict(window=-1), 17),
    (dict(sinks=-1), 17)])
def test_attend_refuses(L, kw, code):
    a = {**ATTEND, **kw}
    _, c = structs(kw)
    assert L.qmv_attend(c, *[a[n] for n in ("q", "out", "ws", "nws", "T", "hq", "qt", "qh", "mn", "ml", "window", "sinks", "scale", "odt")],
                        None) == code


def test_null_structs(L):
    a = [CALL[n] for n in ("q", "kk", "qo", "ko", "T", "hq", "hk", "D", "qt", "qh", "kt", "kh", "xdt", "odt")]
    assert L.qmv_rotate(None, *a, None) == 1
    assert L.qmv_attend_workspace(None, 1, 1, 1, 1, 0, 0) == -1


def tensors(op):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    rot = dict(q=z(3, 8, 64), k=z(3, 2, 64), freqs=torch.zeros(32))
    cache = dict(k_cache=z(5, 16, 2, 64), v_cache=z(5, 16, 2, 64), pages=i(2, 4), starts=i(3), lengths=i(2))
    if op == "rotate":
        return dict(rot, positions=i(3))
    return dict(rot, v=z(3, 2, 64), **cache) if op == "append" else dict(q=z(3, 8, 64), **cache)


F, I = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
BF = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
SHARED = [(dict(eps=-1.0), ValueError, "eps"), (dict(eps=float("nan")), ValueError, "eps"), (dict(eps="a"), TypeError, "eps must be a number"),
          (dict(freqs=BF(32)), TypeError, "freqs must be float32"), (dict(freqs=F(33)), ValueError, "freqs"), (dict(freqs=F(36)), ValueError, "freqs"),
          (dict(freqs=F(30)), ValueError, "multiple of 4"), (dict(positions=F(3)), TypeError, "positions must be int32"),
          (dict(positions=I(4)), ValueError, "positions must be"), (dict(positions=I(2, 3)), ValueError, "need axes"),
          (dict(positions=I(9, 3), axes=I(32)), ValueError, "axes"), (dict(axes=I(31)), ValueError, "axes has shape"),
          (dict(axes=F(32)), TypeError, "axes must be int32"), (dict(q_weight=F(63)), ValueError, "q_weight has shape"),
          (dict(k_weight=F(64).half()), TypeError, "k_weight must be"), (dict(q_weight=F(64), k_weight=BF(64)), TypeError, "share a dtype"),
          (dict(k=F(3, 2, 64)), TypeError, "share a dtype"), (dict(k=BF(4, 2, 64)), ValueError, "k must be"), (dict(k=BF(3, 2, 32)), ValueError, "k must be"),
          (dict(q=F(3, 8, 64).half(), k=F(3, 2, 64).half(), v=F(3, 2, 64).half()), TypeError, "q must be bfloat16 or float32"),
          (dict(q=BF(3, 64, 8).transpose(1, 2)), ValueError, "contiguous"), ({}, ValueError, "CUDA")]
PAGED = [(dict(k_cache=F(5, 16, 2, 64), v_cache=F(5, 16, 2, 64)), TypeError, "k_cache must be"), (dict(v_cache=F(5, 16, 2, 64).half()), TypeError, "share"),
         (dict(v_cache=BF(5, 16, 2, 32)), ValueError, "v_cache has shape"), (dict(k_cache=BF(5, 16, 128)), ValueError, "k_cache must be"),
         (dict(pages=F(2, 4)), TypeError, "pages must be int32"), (dict(pages=I(8)), ValueError, "pages must be"), (dict(starts=I(2)), ValueError, "starts has"),
         (dict(lengths=I(3)), ValueError, "lengths has"), (dict(lengths=I(2).long()), TypeError, "lengths must be int32"),
         (dict(pages=I(4, 2).T), ValueError, "pages: a sequence's"), (dict(q=BF(3, 8, 32)), ValueError, "q must be")]


@pytest.mark.parametrize("op,kw,error,text", [
    *[("rotate", {k: v for k, v in kw.items() if k != "v"}, e, t) for kw, e, t in SHARED], *[("append", *x) for x in SHARED + PAGED],
    *[("attend", *x) for x in PAGED],
    ("rotate", dict(positions=None), ValueError, "positions are missing"), ("rotate", dict(out_dtype=torch.float32), TypeError, "out_dtype"),
    ("rotate", dict(out_dtype=3), TypeError, "out_dtype"), ("append", dict(k=BF(3, 4, 64)), ValueError, "heads"),
    ("append", dict(v=BF(2, 2, 64)), ValueError, "v must be"),
    ("attend", dict(q=F(3, 8, 64)), TypeError, "q must be bfloat16"), ("attend", dict(window=-1), ValueError, "window"),
    ("attend", dict(sinks=-1), ValueError, "sinks"), ("attend", dict(window=1.5), TypeError, "window must be an integer"),
    ("attend", dict(scale=float("inf")), ValueError, "scale"), ("attend", dict(scale="x"), TypeError, "scale must be a number"),
    ("attend", dict(max_new=-1), ValueError, "max_new"), ("attend", dict(max_length="a"), TypeError, "max_length must be an integer"),
    ("attend", {}, ValueError, "CUDA")])
def test_binding_refuses(L, op, kw, error, text):
    import bit_quantized_gemv_amd as q
    with pytest.raises(error, match=text):
        getattr(q, op)(**{**tensors(op), **kw})


@pytest.mark.parametrize("op,kw,text", [("rotate", dict(eps=1e39), "eps"), ("append", dict(eps=4e38), "eps"), ("attend", dict(scale=1e39), "scale"),
                                        ("attend", dict(scale=-3.5e38), "scale")])
def test_binding_refuses_what_fp32_does_not_hold(L, op, kw, text):
    import bit_quantized_gemv_amd as q
    with pytest.raises(ValueError, match=f"{text} must be"):
        getattr(q, op)(**{**tensors(op), **kw})
