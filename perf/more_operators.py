"""What lies between the quantized projections of a decode, verify or prompt
step, as cases that can be timed and compared.

Three operators, each in a plain form (elementary torch operations in 32 bits, or
64 where 32 lose what matters) and as the calls a user makes of the library:

  rotate  norms of queries and keys for each head and their position rotation
          (one axis of positions or several)
  append  the same, with keys and values written into the pages of a cache
  attend  attention of each sequence's new tokens over its pages: causal, with an
          optional sliding window and first tokens that stay visible
"""
import math

import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
MOST_KEYS = 64 * 8192 * 8 * 128      # values of keys that a batch's sequences hold
MOST_PAIRS = 32 * 2048 * 16384       # (head, new token, key)
MOST_VALUES = 8192 * 48 * 128        # values of queries, keys and values of new tokens


def listed():
    return [
        # one token of decode: all latency
        {"name": "append-token", "op": "append", "B": 1, "N": 1, "C": 700, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "R": 128,
         "P": 16, "x": "bf16", "w": "bf16", "y": "bf16", "axes": 1, "far": False, "interleaved": False},
        # verify blocks of several requests in the widest types: fp32 projections, fp16 cache, a part of each head rotated, odd pages
        {"name": "append-odd", "op": "append", "B": 7, "N": 13, "C": 1500, "ragged": True, "Hq": 10, "Hkv": 2, "D": 80, "R": 40,
         "P": 17, "x": "f32", "w": "f32", "y": "f16", "axes": 1, "far": False, "interleaved": True},
        # an image's patches: positions of three axes, no cache
        {"name": "rotate-image", "op": "rotate", "B": 1, "N": 1536, "C": 0, "ragged": False, "Hq": 16, "Hkv": 16, "D": 64, "R": 64,
         "P": 0, "x": "bf16", "w": "none", "y": "bf16", "axes": 3, "far": False, "interleaved": False},
        # prompts that enter a cache
        {"name": "append-prompt", "op": "append", "B": 4, "N": 2048, "C": 2048, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "R": 128,
         "P": 64, "x": "bf16", "w": "bf16", "y": "bf16", "axes": 1, "far": True, "interleaved": False},
        # one token over a short cache: all latency
        {"name": "attend-token", "op": "attend", "B": 1, "N": 1, "C": 411, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 16, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
        # the verify block of one request (13 tokens) over a long document, large heads
        {"name": "attend-verify", "op": "attend", "B": 1, "N": 13, "C": 16384, "ragged": False, "Hq": 16, "Hkv": 8, "D": 256,
         "P": 32, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
        # one token over the longest cache
        {"name": "attend-long", "op": "attend", "B": 1, "N": 1, "C": 131072, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 64, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
        # a serving batch of decode: sequences of very different lengths
        {"name": "attend-batch", "op": "attend", "B": 64, "N": 1, "C": 8192, "ragged": True, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 16, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
        # verify blocks in a layer that sees a window of a long cache and its first tokens
        {"name": "attend-window", "op": "attend", "B": 24, "N": 5, "C": 12000, "ragged": True, "Hq": 16, "Hkv": 4, "D": 64,
         "P": 16, "x": "bf16", "y": "bf16", "window": 1024, "sinks": 4},
        # decode tokens and chunks of prompts in one batch: odd heads, odd pages, fp16 cache, fp32 out
        {"name": "attend-mixed", "op": "attend", "B": 11, "N": 300, "C": 2500, "ragged": True, "Hq": 10, "Hkv": 2, "D": 80,
         "P": 17, "x": "f16", "y": "f32", "window": 700, "sinks": 3},
        # a chunk of a prompt
        {"name": "attend-chunk", "op": "attend", "B": 1, "N": 512, "C": 4096, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 64, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
        # the largest chunk, over a long cache
        {"name": "attend-prompt", "op": "attend", "B": 1, "N": 2048, "C": 16384, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128,
         "P": 64, "x": "bf16", "y": "bf16", "window": 0, "sinks": 0},
    ]


def _log_int(rng, lo, hi):
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "rotate"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    Hq = Hkv * (1 if Hkv == 16 else rng.choice([1, 2, 3, 4, 5, 8] if Hkv <= 4 else [1, 2, 3, 4]))
    D = rng.choice([64, 64, 128, 128, 128, 256, 8 * rng.randint(4, 32)])
    P = rng.choice([16, 16, 32, 64, 256, rng.randint(1, 100)])
    if op != "attend":
        B = 1 if op == "rotate" else _log_int(rng, 1, 64)
        N = _log_int(rng, 1, min(8192, MOST_VALUES // ((Hq + 2 * Hkv) * D * B)))
        axes = rng.choice([1, 2, 3]) if op == "rotate" else rng.choice([1, 1, 3])
        return {"op": op, "B": B, "N": N, "C": 0 if op == "rotate" else N + _log_int(rng, 1, 2000), "ragged": op == "append" and rng.random() < 0.5,
                "Hq": Hq, "Hkv": Hkv, "D": D, "R": rng.choice([D, D, 8 * rng.randint(1, D // 8)]), "P": 0 if op == "rotate" else P,
                "x": rng.choice(["bf16", "bf16", "f32"]), "w": rng.choice(["bf16", "f32", "none"]), "y": rng.choice(["bf16", "bf16", "f16"]),
                "axes": axes, "far": rng.random() < 0.3, "interleaved": rng.random() < 0.3}
    B = _log_int(rng, 1, 64)
    C = _log_int(rng, 16, min(131072, MOST_KEYS // (B * Hkv * D)))
    N = min(C, rng.choice([1, rng.randint(1, 13), _log_int(rng, 1, 2048)]))
    N = max(1, min(N, MOST_PAIRS // (B * Hq * C)))
    window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    return {"op": op, "B": B, "N": N, "C": C, "ragged": rng.random() < 0.6, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P,
            "x": rng.choice(["bf16", "bf16", "f16"]), "y": rng.choice(["bf16", "bf16", "f32"]), "window": window,
            "sinks": rng.choice([0, 4, rng.randint(1, 300)]) if window else 0}


# ---- inputs ---------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _batch(case):
    """How many new tokens each sequence has and how long it is with them. A ragged batch walks from one token to N (a fifth
    of the sequences have all N), and its lengths from the tokens' own number to C."""
    B, N, C = case["B"], case["N"], case["C"]
    if not case["ragged"]:
        return [N] * B, [C] * B
    new = [N if b % 5 == 2 or N == 1 else 1 + (b * 7 + 3) % min(N, 13) for b in range(B)]
    return new, [n + (C - N) * ((b * 11 + 5) % 16) // 15 for b, n in enumerate(new)]


def _cache(g, case, st):
    """Pages of random keys and values in the order of a pool that has been in use; what lies behind a sequence's end was never
    written and holds NaN."""
    B, P, Hkv, D = case["B"], case["P"], case["Hkv"], case["D"]
    new, lengths = _batch(case)
    counts = [-(-n // P) for n in lengths]
    most, total = -(-case["C"] // P) + 1, sum(counts) + 2
    kind = TORCH[case["y"] if case["op"] == "append" else case["x"]]
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([0] + counts, device=DEV).cumsum(0)
    col = torch.arange(most, device=DEV)
    at = first[:-1].unsqueeze(1) + col
    there = col < torch.tensor(counts, device=DEV).unsqueeze(1)
    st["pages"] = torch.where(there, order[at.clamp(max=total - 1)], 0).to(torch.int32)
    st["starts"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    st["lengths"] = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    k = torch.empty(total, P, Hkv, D, device=DEV, dtype=kind)
    v = torch.empty_like(k)
    for t in (k, v):
        for part in t.split(max(1, 2 ** 26 // (P * Hkv * D))):
            part.copy_(_randn(g, *part.shape))
    if case["op"] == "attend":
        last = torch.tensor([n - 1 for n in counts], device=DEV)
        page = st["pages"][torch.arange(B, device=DEV), last].long()
        full = torch.arange(P, device=DEV) < (st["lengths"] - last * P).unsqueeze(1)
        for t in (k, v):
            t[page] = torch.where(full.reshape(B, P, 1, 1), t[page], math.nan)
    st["k_cache"], st["v_cache"] = k, v
    return sum(new)


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = _cache(g, case, st) if case["op"] != "rotate" else case["N"]
    if case["op"] == "attend":
        st["q_in"] = (2.0 * _randn(g, T, Hq, D)).to(TORCH[case["x"]])
        return st
    # one projection's output: queries, keys and values of a token side by side
    qkv = (_randn(g, T, (Hq + 2 * Hkv) * D) * torch.where(_rand(g, (Hq + 2 * Hkv) * D) < 0.02, 8.0, 1.0)).to(TORCH[case["x"]])
    st["q_in"], st["k_in"], st["v_in"] = (p.unflatten(1, (-1, D)) for p in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
    half = case["R"] // 2
    st["freqs"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
    A = case["axes"]
    st["axis"] = None if A == 1 else (torch.arange(half, device=DEV) % A).to(torch.int32)
    top = 2 ** 20 if case["far"] else 4096
    given = case["op"] == "rotate" or A > 1 or case["far"]
    st["positions"] = torch.randint(0, top, (A, T), generator=g, device=DEV, dtype=torch.int32) if given else None
    for n in ("q", "k"):
        st[n + "_weight"] = None if case["w"] == "none" else (1.0 + 0.3 * _randn(g, D)).to(TORCH[case["w"]])
    return st


# ---- the plain forms ------------------------------------------------------


def _turn_plain(x, weight, cos, sin, interleaved):
    """Norm and rotation of [T][H][D] in 32 bits; cos, sin: [T][1][R/2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _places(st):
    """Each token's sequence, and its place in it."""
    t = torch.arange(st["q_in"].shape[0], device=DEV)
    b = (t.unsqueeze(1) >= st["starts"][1:]).sum(1)
    first = st["lengths"] - (st["starts"][1:] - st["starts"][:-1])
    return b, first[b] + t - st["starts"][b]


def _rotate_plain(st):
    positions = st["positions"]
    if st["op"] == "append":
        b, place = _places(st)
    if positions is None:
        positions = place.unsqueeze(0)
    axis = torch.zeros_like(st["freqs"]).long() if st["axis"] is None else st["axis"].long()
    angle = positions.T[:, axis].double() * st["freqs"].double()        # far positions: 64 bits
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    kind = TORCH[st["y"]]
    q = _turn_plain(st["q_in"], st["q_weight"], cos, sin, st["interleaved"]).to(kind)
    k = _turn_plain(st["k_in"], st["k_weight"], cos, sin, st["interleaved"]).to(kind)
    if st["op"] == "rotate":
        return {"q": q, "k": k}
    page, slot = st["pages"][b, place // st["P"]].long(), place % st["P"]
    st["k_cache"][page, slot] = k
    st["v_cache"][page, slot] = st["v_in"].to(kind)
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _attend_plain(st):
    B, N, C, P, Hq, Hkv, D = (st[n] for n in ("B", "N", "C", "P", "Hq", "Hkv", "D"))
    b, place = _places(st)
    row = torch.arange(b.shape[0], device=DEV) - st["starts"][b]
    new = st["starts"][1:] - st["starts"][:-1]
    i, j = torch.arange(N, device=DEV), torch.arange(C, device=DEV)
    q = st["q_in"][(st["starts"][:-1].unsqueeze(1) + i).clamp(max=b.shape[0] - 1)].float()
    q = q.reshape(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    page, slot = st["pages"][:, j // P].long(), j % P
    held = (j < st["lengths"].unsqueeze(1)).reshape(B, C, 1, 1)
    k = torch.where(held, st["k_cache"][page, slot], 0.0).float().permute(0, 2, 3, 1)
    s = torch.matmul(q, k).reshape(B, Hkv, Hq // Hkv, N, C) * (1.0 / math.sqrt(D))
    del k
    at = ((st["lengths"] - new).unsqueeze(1) + i).unsqueeze(-1)
    sees = j <= at
    if st["window"]:
        sees = sees & ((j > at - st["window"]) | (j < st["sinks"]))
    s = s.masked_fill_(~sees.reshape(B, 1, 1, N, C), -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp_(s.sub_(torch.where(top > -math.inf, top, 0.0)))
    total = e.sum(-1).reshape(B, Hkv, -1, 1)
    v = torch.where(held, st["v_cache"][page, slot], 0.0).float().transpose(1, 2)
    o = torch.matmul(e.reshape(B, Hkv, -1, C), v) / torch.where(total > 0, total, 1.0)
    o = o.reshape(B, Hkv, Hq // Hkv, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    return {"o": o[b, row].to(TORCH[st["y"]])}


def run(st):
    if own:
        import bit_quantized_gemv_amd as q
        if st["op"] == "attend":
            return {"o": q.attend(st["q_in"], st["k_cache"], st["v_cache"], st["pages"], st["starts"], st["lengths"],
                                  window=st["window"], sinks=st["sinks"], max_new=st["N"], max_length=st["C"],
                                  out_dtype=TORCH[st["y"]])}
        how = {"q_weight": st["q_weight"], "k_weight": st["k_weight"], "eps": EPS, "axes": st["axis"], "interleaved": st["interleaved"]}
        if st["op"] == "rotate":
            y, k = q.rotate(st["q_in"], st["k_in"], st["freqs"], st["positions"], out_dtype=TORCH[st["y"]], **how)
            return {"q": y, "k": k}
        y = q.append(st["q_in"], st["k_in"], st["v_in"], st["freqs"], st["k_cache"], st["v_cache"], st["pages"], st["starts"],
                     st["lengths"], positions=st["positions"], **how)
        return {"q": y, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return _attend_plain(st) if st["op"] == "attend" else _rotate_plain(st)


# ---- what a pass cannot do without ----------------------------------------


def _visible(case, place):
    """How many keys a token at this place sees."""
    if not case["window"]:
        return place + 1
    low = max(0, place - case["window"] + 1)
    return place + 1 - low + min(low, case["sinks"])


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, lengths = ([case["N"]], [0]) if case["op"] == "rotate" else _batch(case)
    T = sum(new)
    if case["op"] != "attend":
        heads = Hq + (2 if case["op"] == "append" else 1) * Hkv
        return {"bytes": T * heads * D * (SIZE[case["x"]] + SIZE[case["y"]]) + T * 4 * case["axes"], "flops": 10.0 * T * heads * D}
    keys = pairs = 0
    for n, length in zip(new, lengths):
        pairs += sum(_visible(case, length - n + i) for i in range(n))
        low = max(0, length - n - case["window"] + 1) if case["window"] else 0
        keys += length - low + min(low, case["sinks"])
    return {"bytes": keys * Hkv * D * 2 * SIZE[case["x"]] + T * Hq * D * (SIZE[case["x"]] + SIZE[case["y"]]),
            "flops": 4.0 * D * Hq * pairs}


# ---- the definitions in 64 bits -------------------------------------------


def _turned64(x, weight, angles, interleaved):
    """Each pair of values as a complex number, turned by its angle."""
    x = x.double()
    if weight is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** 0.5 * weight.double()
    half = angles.shape[-1]
    first = torch.arange(half, device=DEV) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angles), angles).unsqueeze(1)
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    new, lengths = ([case["N"]], [case["N"]]) if case["op"] == "rotate" else _batch(case)
    places = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lengths)]).to(DEV)
    if case["op"] != "attend":
        pos = places.unsqueeze(0) if st["positions"] is None else st["positions"]
        rows = pos[[0] * (case["R"] // 2) if st["axis"] is None else st["axis"].tolist()]
        angles = rows.T.double() * st["freqs"].double()
        q, k = (_turned64(st[n + "_in"], st[n + "_weight"], angles, case["interleaved"]) for n in ("q", "k"))
        if case["op"] == "rotate":
            return {"q": q, "k": k}
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        begin = 0
        for b, (m, n) in enumerate(zip(new, lengths)):
            j = torch.arange(n - m, n, device=DEV)
            rows = st["pages"][b].long()[j // case["P"]] * case["P"] + j % case["P"]
            kc.view(-1, Hkv, D)[rows] = k[begin:begin + m]
            vc.view(-1, Hkv, D)[rows] = st["v_in"][begin:begin + m].double()
            begin += m
        return {"q": q, "k_cache": kc, "v_cache": vc}
    o = torch.zeros(sum(new), Hq, D, dtype=torch.float64, device=DEV)
    begin = 0
    for b, (m, n) in enumerate(zip(new, lengths)):
        count = -(-n // case["P"])
        for h in range(Hkv):
            k, v = (st[c][st["pages"][b, :count].long(), :, h].flatten(0, 1)[:n].double() for c in ("k_cache", "v_cache"))
            for i in range(0, m, 512):
                e = min(m, i + 512)
                q = st["q_in"][begin + i:begin + e, h * G:(h + 1) * G].double()
                s = torch.matmul(q.reshape(-1, D), k.T).reshape(e - i, G, n) / D ** 0.5
                gap = torch.arange(n - m + i, n - m + e, device=DEV).unsqueeze(1) - torch.arange(n, device=DEV)
                hidden = gap < 0
                if case["window"]:
                    hidden = hidden | ((gap >= case["window"]) & (torch.arange(n, device=DEV) >= case["sinks"]))
                p = torch.softmax(s.masked_fill(hidden.unsqueeze(1), -math.inf), -1)
                o[begin + i:begin + e, h * G:(h + 1) * G] = torch.matmul(p.reshape(-1, n), v).reshape(e - i, G, D)
        begin += m
    return {"o": o}
