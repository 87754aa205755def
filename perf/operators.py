"""The operators of a decode or verify step that stand beside the quantized
product, as cases that can be timed and compared.

Three operators, each in a plain form (elementary torch operations in 32 bits,
or 64 where 32 lose what matters) and as the calls a user makes of the library:

  lora    y[m] = W x[m] + c_a B_a (A_a x[m]), a = ids[m]: the affine-quantized
          projection of many requests' tokens, each with its own low-rank
          adapter (or none)
  moe     a mixture-of-experts layer for a few tokens: router product, top-k
          and softmax, then the chosen affine-quantized experts' gated product
          and their weighted sum
  verify  accept or replace drafted tokens by the target's probabilities and
          given random numbers
"""
import math

import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LARGEST = {"lora": 17408 * 5120, "moe": 128 * 2048 * 1024, "verify": 32 * 8 * 131072}


def listed():
    return [
        # one token of one request on the up projection of a 12B-class model: the decode step with an adapter
        {"name": "lora-decode", "op": "lora", "M": 1, "N": 15360, "K": 3840, "bits": 4, "gs": 64, "x": "bf16",
         "sb": "bf16", "y": "bf16", "R": 16, "L": 8, "ad": "bf16", "mix": False},
        # the verify block of one request (13 tokens, one adapter) on the down projection
        {"name": "lora-verify", "op": "lora", "M": 13, "N": 3840, "K": 15360, "bits": 4, "gs": 64, "x": "bf16",
         "sb": "bf16", "y": "bf16", "R": 32, "L": 4, "ad": "bf16", "mix": False},
        # a small odd projection in the library's widest types: fp32 in and out, fp16 scales, 2-bit codes, a rank that fills no tile
        {"name": "lora-odd", "op": "lora", "M": 5, "N": 1001, "K": 1344, "bits": 2, "gs": 64, "x": "f32",
         "sb": "f16", "y": "f32", "R": 5, "L": 3, "ad": "f16", "mix": True},
        # a serving batch of 64 requests over 32 adapters, some with none, on the up projection of a 27B-class model
        {"name": "lora-batch", "op": "lora", "M": 64, "N": 17408, "K": 5120, "bits": 4, "gs": 64, "x": "bf16",
         "sb": "bf16", "y": "bf16", "R": 64, "L": 32, "ad": "bf16", "mix": True},
        # a toy layer: what a test or a small draft model runs, all launch latency
        {"name": "moe-small", "op": "moe", "T": 3, "E": 7, "k": 2, "D": 320, "F": 192, "bits": 4, "gs": 64,
         "x": "f32", "sb": "f16", "y": "f32", "renorm": False},
        # one token of decode
        {"name": "moe-decode", "op": "moe", "T": 1, "E": 64, "k": 6, "D": 3840, "F": 1024, "bits": 4, "gs": 64,
         "x": "bf16", "sb": "bf16", "y": "bf16", "renorm": True},
        # a verify block of 13 tokens over many experts: most experts meet one token or two
        {"name": "moe-verify", "op": "moe", "T": 13, "E": 128, "k": 8, "D": 2048, "F": 1024, "bits": 4, "gs": 64,
         "x": "bf16", "sb": "bf16", "y": "bf16", "renorm": True},
        # a serving batch: every expert is met, by about 16 tokens; 2-bit codes in groups of 128
        {"name": "moe-batch", "op": "moe", "T": 128, "E": 32, "k": 4, "D": 3840, "F": 1920, "bits": 2, "gs": 128,
         "x": "bf16", "sb": "bf16", "y": "bf16", "renorm": True},
        # one request, one drafted token, a small vocabulary in fp32, a drafter that gives tokens only
        {"name": "verify-small", "op": "verify", "B": 1, "S": 1, "V": 32000, "logits": "f32", "probs": "none",
         "temp": "one", "ragged": False, "masked": False},
        # one request's draft block of five positions at a large vocabulary
        {"name": "verify-block", "op": "verify", "B": 1, "S": 4, "V": 131072, "logits": "bf16", "probs": "f32",
         "temp": "one", "ragged": False, "masked": False},
        # requests with drafts of different lengths and temperatures (some greedy), part of the vocabulary masked by a grammar
        {"name": "verify-ragged", "op": "verify", "B": 13, "S": 12, "V": 50001, "logits": "f32", "probs": "bf16",
         "temp": "mixed", "ragged": True, "masked": True},
        # a serving batch
        {"name": "verify-batch", "op": "verify", "B": 32, "S": 7, "V": 131072, "logits": "bf16", "probs": "f32",
         "temp": "mixed", "ragged": False, "masked": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "moe", "verify"])
    bits, gs = rng.choice([4, 4, 4, 2]), rng.choice([64, 64, 128])
    types = {"x": rng.choice(["bf16", "bf16", "f32"]), "sb": rng.choice(["bf16", "f16"]), "y": rng.choice(["bf16", "f32"])}
    if op == "lora":
        N = _log_int(rng, 64, 17408)
        K = gs * _log_int(rng, 1, min(17408, LARGEST["lora"] // N) // gs)
        return {"op": op, "M": _log_int(rng, 1, 64), "N": N, "K": K, "bits": bits, "gs": gs, **types,
                "R": rng.choice([rng.randint(1, 64), 8, 16, 32, 64]), "L": _log_int(rng, 1, 32),
                "ad": rng.choice(["bf16", "bf16", "f16"]), "mix": rng.random() < 0.7}
    if op == "moe":
        E = _log_int(rng, 4, 128)
        D = gs * _log_int(rng, 1, 3840 // gs)
        F = gs * _log_int(rng, 1, min(2048, LARGEST["moe"] // (E * D)) // gs)
        return {"op": op, "T": _log_int(rng, 1, 128), "E": E, "k": rng.randint(1, min(8, E)), "D": D, "F": F,
                "bits": bits, "gs": gs, **types, "renorm": rng.random() < 0.7}
    V = _log_int(rng, 1000, 262144)
    S = rng.randint(0, 12)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(64, LARGEST["verify"] // (V * (S + 1))))), "S": S, "V": V,
            "logits": rng.choice(["bf16", "f32"]), "probs": rng.choice(["f32", "bf16", "none"]),
            "temp": rng.choice(["one", "mixed"]), "ragged": rng.random() < 0.5, "masked": rng.random() < 0.3}


# ---- inputs ---------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _weights(g, lead, K, bits, gs, sb):
    """Packed codes (uniform), scales for weights of about unit gain, and biases near the middle of the codes' range."""
    w = torch.randint(-2 ** 31, 2 ** 31, (*lead, K * bits // 32), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    top = 2 ** bits - 1
    spread = math.sqrt(((top + 1) ** 2 - 1) / 12.0)
    s = (0.5 + _rand(g, *lead, K // gs)) / (spread * math.sqrt(K))
    b = -s * (0.5 * top + 0.25 * _randn(g, *lead, K // gs))
    return w, s.to(TORCH[sb]).contiguous(), b.to(TORCH[sb]).contiguous()


def _hidden(g, T, D, kind):
    """Activations: normal, with a few channels that stand out tenfold in all tokens."""
    loud = torch.where(_rand(g, D) < 0.01, 10.0, 1.0)
    return (_randn(g, T, D) * loud).to(TORCH[kind])


def _ids(case):
    """Which adapter each token uses: one request's tokens share one; a mixed batch walks over all of them and -1 (none)."""
    m = torch.arange(case["M"], dtype=torch.int32)
    return (m * 5 + 1) % (case["L"] + 1) - 1 if case["mix"] else torch.full_like(m, case["L"] // 2)


def _lengths(case):
    """How many drafted tokens each request has."""
    b = torch.arange(case["B"], dtype=torch.int32)
    return (b * 7 + 3) % (case["S"] + 1) if case["ragged"] else torch.full_like(b, case["S"])


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    if case["op"] == "lora":
        M, N, K, R, L = case["M"], case["N"], case["K"], case["R"], case["L"]
        st["w"], st["s"], st["b"] = _weights(g, (N,), K, case["bits"], case["gs"], case["sb"])
        st["inp"] = _hidden(g, M, K, case["x"])
        st["la"] = (_randn(g, L, R, K) / math.sqrt(K)).to(TORCH[case["ad"]])
        st["lb"] = (_randn(g, L, N, R) * 0.3 / math.sqrt(R)).to(TORCH[case["ad"]])
        st["scaling"] = 0.5 + 1.5 * _rand(g, L)
        st["ids"] = _ids(case).to(DEV)
    elif case["op"] == "moe":
        T, E, D, F = case["T"], case["E"], case["D"], case["F"]
        st["inp"] = _hidden(g, T, D, case["x"])
        st["router"] = (_randn(g, E, D) / math.sqrt(D)).to(TORCH[case["x"]])
        st["w13"], st["s13"], st["b13"] = _weights(g, (E, 2 * F), D, case["bits"], case["gs"], case["sb"])
        st["w2"], st["s2"], st["b2"] = _weights(g, (E, D), F, case["bits"], case["gs"], case["sb"])
    else:
        B, S, V = case["B"], case["S"], case["V"]
        peaks = torch.where(_rand(g, B, S + 1, V) < 20.0 / V, 7.0, 0.0)
        logits = 2.0 * _randn(g, B, S + 1, V) + peaks
        if case["masked"]:
            gone = (_rand(g, B, 1, V) < 0.9) & (torch.arange(B, device=DEV) % 2 == 0).reshape(B, 1, 1)
            logits = torch.where(gone, -math.inf, logits)
        st["logits_in"] = logits.to(TORCH[case["logits"]])
        temp = torch.ones(B, device=DEV)
        if case["temp"] == "mixed":
            temp = 0.3 + 0.9 * _rand(g, B)
            temp[2::4] = 0.0
        st["temperature"] = temp
        # the drafter: a noisy copy of the target
        drafter = logits[:, :S] + 0.7 * _randn(g, B, S, V)
        if case["probs"] == "none":
            st["draft"], st["q"] = drafter.argmax(-1).to(torch.int32), None
        else:
            q = torch.softmax(drafter, -1).to(TORCH[case["probs"]])
            c = q.double().cumsum(-1)
            at = _rand(g, B, S, 1).double() * c[..., -1:]
            st["draft"] = torch.searchsorted(c, at, right=True).squeeze(-1).clamp(max=V - 1).to(torch.int32)
            st["q"] = q
        st["u"] = _rand(g, B, S + 1)
        st["lengths"] = _lengths(case).to(DEV)
    return st


# ---- the plain forms ------------------------------------------------------


def _dequantize(w, s, b, bits, gs):
    """scale * code + bias for the last axis, in 32 bits."""
    shifts = torch.arange(0, 32, bits, device=w.device, dtype=torch.int32)
    codes = (w.unsqueeze(-1) >> shifts) & (2 ** bits - 1)
    codes = codes.reshape(*s.shape, gs).float()
    return (codes * s.float().unsqueeze(-1) + b.float().unsqueeze(-1)).reshape(*w.shape[:-1], -1)


def _lora_plain(st):
    x = st["inp"].float()
    y = x @ _dequantize(st["w"], st["s"], st["b"], st["bits"], st["gs"]).T
    has = st["ids"] >= 0
    a = st["ids"].clamp(min=0).long()
    h = torch.matmul(st["la"][a].float(), x.unsqueeze(-1))
    d = torch.matmul(st["lb"][a].float(), h).squeeze(-1) * st["scaling"][a].unsqueeze(-1)
    return {"y": (y + torch.where(has.unsqueeze(-1), d, 0.0)).to(TORCH[st["y"]])}


def _route_plain(x, router, k, renorm):
    """The k largest router products of each token (ties to the lowest index) and their softmax weights, in 64 bits: near
    ties are decided as the exact products would."""
    logits = x.double() @ router.double().T
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    weights = torch.softmax(top, -1)[:, :k]
    if renorm:
        weights = torch.softmax(top[:, :k], -1)
    return weights.float(), ids[:, :k].to(torch.int32)


def _moe_plain(st):
    T, E, k, F = st["T"], st["E"], st["k"], st["F"]
    weights, ids = _route_plain(st["inp"], st["router"], k, st["renorm"])
    pick = ids.reshape(-1).long()
    x = st["inp"].float()
    few = T * k < E
    used = pick if few else torch.arange(E, device=x.device)
    w13 = _dequantize(st["w13"][used], st["s13"][used], st["b13"][used], st["bits"], st["gs"])
    xs = x.repeat_interleave(k, 0).unsqueeze(1) if few else x.unsqueeze(0).expand(E, -1, -1)
    gu = torch.matmul(xs, w13.transpose(1, 2))
    gate, up = gu[..., :F], gu[..., F:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    del w13, gu
    w2 = _dequantize(st["w2"][used], st["s2"][used], st["b2"][used], st["bits"], st["gs"])
    z = torch.matmul(h, w2.transpose(1, 2))
    if few:
        z = z.reshape(T, k, -1)
    else:
        z = z[ids.long(), torch.arange(T, device=x.device).unsqueeze(-1)]
    y = (z * weights.unsqueeze(-1)).sum(1)
    return {"y": y.to(TORCH[st["y"]]), "weights": weights, "ids": ids}


def _first(hit):
    """The lowest index along the last axis where `hit` holds (the axis's length if none does)."""
    V = hit.shape[-1]
    return torch.where(hit, torch.arange(V, device=hit.device), V).amin(-1)


def _verify_plain(st):
    """In 64 bits: which token a cumulative sum first passes a given number at is decided by small differences."""
    B, S, V = st["B"], st["S"], st["V"]
    dev = st["u"].device
    l = st["logits_in"].double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    top = l.amax(-1, keepdim=True)
    live = l > -math.inf
    T = st["temperature"].double().reshape(B, 1, 1)
    e = torch.exp((l - top) / torch.where(T > 0, T, 1.0))
    e = torch.where(l == top, 1.0, e)
    at_top = torch.arange(V, device=dev) == _first(l == top).unsqueeze(-1)
    e = torch.where(live, torch.where(T > 0, e, at_top.double()), 0.0)
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    drafts, rows = st["draft"].long(), torch.arange(B, device=dev)
    lens = st["lengths"].long()
    if S:
        px = p[:, :S].gather(-1, drafts.unsqueeze(-1)).squeeze(-1)
        qx = torch.ones_like(px) if st["q"] is None else st["q"].gather(-1, drafts.unsqueeze(-1)).squeeze(-1).double()
        yes = (st["u"][:, :S].double() * qx < px) & (torch.arange(S, device=dev) < lens.unsqueeze(-1))
        n = yes.long().cumprod(-1).sum(-1)
    else:
        n = torch.zeros(B, dtype=torch.long, device=dev)
    p_n = p[rows, n]
    weight = p_n
    if S:
        at = n.clamp(max=S - 1)
        if st["q"] is None:
            q_n = (torch.arange(V, device=dev) == drafts[rows, at].unsqueeze(-1)).double()
        else:
            q_n = st["q"][rows, at].double()
        rest = (p_n - q_n).clamp(min=0.0)
        use = ((n < lens) & (rest.sum(-1) > 0)).unsqueeze(-1)
        weight = torch.where(use, rest, p_n)
    c = weight.cumsum(-1)
    u_last = st["u"].double()[rows, lens]
    new = _first(c > (u_last * c[:, -1]).unsqueeze(-1))
    last = V - 1 - _first((weight > 0).flip(-1))
    new = torch.where(new < V, new, last)
    j = torch.arange(S + 1, device=dev)
    padded = torch.cat([drafts, torch.zeros(B, 1, dtype=torch.long, device=dev)], 1)
    tokens = torch.where(j < n.unsqueeze(-1), padded, torch.where(j == n.unsqueeze(-1), new.unsqueeze(-1), -1))
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32)}


def run(st):
    if own:
        import bit_quantized_gemv_amd as q
        if st["op"] == "lora":
            return {"y": q.affine_lora(st["w"], st["s"], st["b"], st["inp"], st["la"], st["lb"], st["ids"],
                                       scaling=st["scaling"], bits=st["bits"], group_size=st["gs"],
                                       out_dtype=TORCH[st["y"]])}
        if st["op"] == "moe":
            y, weights, ids = q.moe(st["inp"], st["router"], (st["w13"], st["s13"], st["b13"]),
                                    (st["w2"], st["s2"], st["b2"]), top_k=st["k"], bits=st["bits"],
                                    group_size=st["gs"], renormalize=st["renorm"], out_dtype=TORCH[st["y"]],
                                    return_routing=True)
            return {"y": y, "weights": weights, "ids": ids}
        tokens, accepted = q.verify(st["logits_in"], st["draft"], st["u"], draft_probs=st["q"],
                                    temperature=st["temperature"], lengths=st["lengths"])
        return {"tokens": tokens, "accepted": accepted}
    return {"lora": _lora_plain, "moe": _moe_plain, "verify": _verify_plain}[st["op"]](st)


# ---- what a pass cannot do without ----------------------------------------

SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    if case["op"] == "lora":
        M, N, K, R = case["M"], case["N"], case["K"], case["R"]
        used = set(_ids(case).tolist())
        tokens = sum(i >= 0 for i in _ids(case).tolist())
        adapters = len(used - {-1})
        nbytes = N * K * case["bits"] / 8 + N * (K // case["gs"]) * 4 + M * K * SIZE[case["x"]] + M * N * SIZE[case["y"]]
        return {"bytes": nbytes + adapters * R * (K + N) * 2 + M * 4, "flops": 2.0 * M * N * K + 2.0 * tokens * R * (K + N)}
    if case["op"] == "moe":
        T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
        met = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens choose, if all are alike
        expert = 3 * D * F * (case["bits"] / 8 + 4 / case["gs"])
        nbytes = met * expert + E * D * SIZE[case["x"]] + T * D * (SIZE[case["x"]] + SIZE[case["y"]]) + T * k * 8
        return {"bytes": nbytes, "flops": 6.0 * T * k * D * F + 2.0 * T * E * D}
    # every position's logits once; the drafter's probabilities of the one position that is sampled again
    B, V = case["B"], case["V"]
    rows = int(_lengths(case).sum()) + B
    nbytes = rows * V * SIZE[case["logits"]] + (0 if case["probs"] == "none" else B * V * SIZE[case["probs"]] if case["S"] else 0)
    return {"bytes": nbytes + B * (case["S"] + 1) * 12, "flops": 4.0 * rows * V + 4.0 * B * V}


# ---- the definitions in 64 bits -------------------------------------------


def _fields(w, bits):
    """The codes of packed words, by bytes: low fields first."""
    by = w.contiguous().view(torch.uint8)
    parts = [(by // 2 ** s) % 2 ** bits for s in range(0, 8, bits)]
    return torch.stack(parts, -1).reshape(*w.shape[:-1], -1)


def _product64(x, w, s, b, bits, gs):
    """sum over groups of scale * sum(code * x) + bias * sum(x), in 64 bits, rows in pieces."""
    T, K = x.shape
    G = K // gs
    xg = x.double().reshape(T, G, gs)
    sums = xg.sum(-1)
    out = torch.empty(T, w.shape[0], dtype=torch.float64, device=x.device)
    step = max(1, 2 ** 24 // max(1, T * G))
    for n in range(0, w.shape[0], step):
        c = _fields(w[n:n + step], bits).double().reshape(-1, G, gs)
        dots = torch.matmul(xg.transpose(0, 1), c.permute(1, 2, 0))  # [G, T, rows]
        out[:, n:n + step] = (dots * s[n:n + step].double().T.unsqueeze(1)).sum(0) + sums @ b[n:n + step].double().T
    return out


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "lora":
        y = _product64(st["inp"], st["w"], st["s"], st["b"], case["bits"], case["gs"])
        for m, a in enumerate(st["ids"].tolist()):
            if a >= 0:
                h = st["la"][a].double() @ st["inp"][m].double()
                y[m] += st["scaling"][a].double() * (st["lb"][a].double() @ h)
        return {"y": y}
    F, k = case["F"], case["k"]
    x = st["inp"].double()
    scores = x @ st["router"].double().T
    rows = [sorted(range(case["E"]), key=lambda e: (-r[e], e))[:k] for r in scores.tolist()]
    ids = torch.tensor(rows, device=x.device)
    chosen = torch.exp(scores.gather(1, ids) - scores.amax(1, keepdim=True))
    weights = chosen / (chosen if case["renorm"] else torch.exp(scores - scores.amax(1, keepdim=True))).sum(1, keepdim=True)
    y = torch.zeros(case["T"], case["D"], dtype=torch.float64, device=x.device)
    for e in sorted({e for r in rows for e in r}):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = _product64(x[t], st["w13"][e], st["s13"][e], st["b13"][e], case["bits"], case["gs"])
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        z = _product64(h, st["w2"][e], st["s2"][e], st["b2"][e], case["bits"], case["gs"])
        y.index_add_(0, t, z * weights[t, j].unsqueeze(-1))
    return {"y": y, "weights": weights, "ids": None}
