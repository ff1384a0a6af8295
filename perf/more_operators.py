"""What is measured of the operators around a cache held in 8 bits and of beam search over it: new keys and values
rotated, quantised and written; cached tokens read back; attention of new tokens over the quantised cache; the selection
of the next beams among beams and vocabulary; and the reordering of the beams' block tables with the copies it needs.
``run`` computes each in elementary torch operations, or, with ``own``, through ``certified_fixed_stabilizer_gb300.clis``.

A quantised row (one token and key/value head) is d codes and one fp32 scale: the row's largest magnitude over 127
(int8) or 448 (E4M3), and each value over the scale, rounded to the nearest code.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100  # a row whose largest magnitude is below this is held as zeros


# ------------------------------------------------------------------- cases


def listed():
    return [
        # New keys and values of 64 decoding requests, written and looked at again: latency alone.
        {"name": "store_decode", "op": "store", "S": 64, "new": 1, "chunks": 0, "ctx": 4000, "H": 32, "Hk": 8, "d": 128,
         "page": 16, "pairs": 64, "axes": 1, "interleaved": False, "dtype": "bf16", "code": "int8", "lens": 1},
        # A prompt's chunk with video positions, written and read back for a dense call.
        {"name": "store_chunk", "op": "store", "S": 1, "new": 8192, "chunks": 1, "ctx": 1000, "H": 32, "Hk": 8, "d": 128,
         "page": 64, "pairs": 64, "axes": 3, "interleaved": True, "dtype": "fp16", "code": "e4m3", "lens": 2},
        # Three short sequences read back: latency alone.
        {"name": "read_few", "op": "read", "S": 3, "ctx": 71, "Hk": 4, "d": 64, "page": 16, "dtype": "fp16",
         "code": "e4m3", "lens": 3},
        # Long sequences read back, as for a move to another cache: the bytes.
        {"name": "read_long", "op": "read", "S": 8, "ctx": 30011, "Hk": 8, "d": 128, "page": 64, "dtype": "bf16",
         "code": "int8", "lens": 4},
        # One request, a short cache: latency alone.
        {"name": "attn_one", "op": "attn", "S": 1, "new": 1, "chunks": 0, "ctx": 300, "even": True, "H": 32, "Hk": 8,
         "d": 128, "page": 16, "causal": True, "dtype": "bf16", "code": "int8", "lens": 5},
        # Single tokens of 64 requests of very different lengths: the cache's bytes.
        {"name": "attn_decode", "op": "attn", "S": 64, "new": 1, "chunks": 0, "ctx": 16000, "even": False, "H": 32,
         "Hk": 8, "d": 128, "page": 16, "causal": True, "dtype": "bf16", "code": "int8", "lens": 6},
        # Drafted tokens (up to 5 a request, 8 query heads to a key/value head): 40 rows over the same keys.
        {"name": "attn_draft", "op": "attn", "S": 17, "new": 5, "chunks": 17, "ctx": 9001, "even": False, "H": 32,
         "Hk": 4, "d": 128, "page": 64, "causal": True, "dtype": "fp16", "code": "e4m3", "lens": 7},
        # A chunk of a long prompt behind 30,000 cached tokens: the tensor cores.
        {"name": "attn_chunk", "op": "attn", "S": 1, "new": 2048, "chunks": 1, "ctx": 30011, "even": True, "H": 32,
         "Hk": 8, "d": 128, "page": 64, "causal": True, "dtype": "bf16", "code": "int8", "lens": 8},
        # The next token of 8 requests of 4 beams, an odd vocabulary, twice as many candidates as beams.
        {"name": "beam_few", "op": "beam", "R": 8, "W": 4, "V": 32003, "K": 8, "dtype": "bf16", "masked": False, "dead": False},
        # A large batch and vocabulary, a fifth of the words masked, some beams not in use: the bytes of the logits.
        {"name": "beam_many", "op": "beam", "R": 96, "W": 8, "V": 128000, "K": 16, "dtype": "bf16", "masked": True, "dead": True},
        # One step of 8 requests of 4 beams, a cache of 16-bit values: latency alone.
        {"name": "reorder_few", "op": "reorder", "R": 8, "W": 4, "ctx": 1000, "tail": 60, "layers": 2, "Hk": 8, "d": 128,
         "page": 16, "dtype": "bf16", "code": "", "ended": False, "lens": 9},
        # 64 requests of 8 beams, pages of 64 tokens in 8 bits with scales, some requests at their end.
        {"name": "reorder_many", "op": "reorder", "R": 64, "W": 8, "ctx": 8000, "tail": 200, "layers": 4, "Hk": 8, "d": 128,
         "page": 64, "dtype": "bf16", "code": "int8", "ended": True, "lens": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attn", "attn", "attn", "beam", "beam", "reorder"])
    dtype, code = rng.choice(["bf16", "fp16"]), rng.choice(["int8", "e4m3"])
    if op == "beam":
        R, W = _log(rng, 1, 96), _log(rng, 1, 16)
        V = _log(rng, 1, max(1, min(200000, 90000000 // (R * W))))
        return {"op": "beam", "R": R, "W": W, "V": V, "K": rng.randint(1, 2 * W), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "masked": rng.random() < 0.5, "dead": rng.random() < 0.5}
    d, Hk = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    page, lens = rng.choice([8, 16, 32, 64, 128]), rng.randrange(1 << 20)
    if op == "reorder":
        return {"op": "reorder", "R": _log(rng, 1, 64), "W": rng.randint(1, 8), "ctx": _log(rng, 1, 8000),
                "tail": _log(rng, 1, 200), "layers": rng.randint(1, 3), "Hk": Hk, "d": d, "page": min(page, 64), "dtype": dtype,
                "code": rng.choice(["", "int8", "e4m3"]), "ended": rng.random() < 0.5, "lens": lens}
    if op == "read":
        return {"op": "read", "S": _log(rng, 1, 64), "ctx": _log(rng, 1, 4000), "Hk": Hk, "d": d, "page": page,
                "dtype": dtype, "code": code, "lens": lens}
    H = Hk * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "store":
        axes = rng.choice([1, 2, 3, 4])
        pairs = rng.choice([p for p in (8, 16, 24, 32, 48, 64) if p <= d // 2])
        S = _log(rng, 1, 64)
        return {"op": "store", "S": S, "new": _log(rng, 1, 8192 // S), "chunks": rng.randint(0, S), "ctx": _log(rng, 1, 4000),
                "H": H, "Hk": Hk, "d": d, "page": page, "pairs": pairs, "axes": axes, "interleaved": rng.random() < 0.5,
                "dtype": dtype, "code": code, "lens": lens}
    # attention: single and drafted tokens over many caches, or chunks; rows times keys stay under the listed ones'.
    if rng.random() < 0.6:
        S, new = _log(rng, 1, 64), _log(rng, 1, 8)
        ctx, chunks = _log(rng, 1, 16000), rng.randint(0, S)
    else:
        S, new = rng.randint(1, 6), _log(rng, 9, 1024)
        ctx, chunks = _log(rng, 1, 8000), rng.randint(1, S)
    return {"op": "attn", "S": S, "new": new, "chunks": chunks, "ctx": ctx, "even": rng.random() < 0.3, "H": H, "Hk": Hk,
            "d": d, "page": page, "causal": rng.random() < 0.8, "dtype": dtype, "code": code, "lens": lens}


def _lengths(case):
    """(cached, new) lengths of a case's sequences."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for s in range(case["S"]):
        ctx.append(case["ctx"] if case.get("even") else rng.randint(case["ctx"] // 16, case["ctx"]))
        new.append(0 if "new" not in case else 1 if s >= case["chunks"] else case["new"] if s == 0 else rng.randint(1, case["new"]))
    return ctx, new


def _beams(case):
    """Of each request: tokens that its beams share, further tokens of each beam (or none: at its end)."""
    rng = random.Random(case["lens"])
    got = []
    for r in range(case["R"]):
        shared, tail = rng.randint(case["ctx"] // 16, case["ctx"]), rng.randint(1, case["tail"])
        parent = [rng.randrange(case["W"]) for _ in range(case["W"])]
        if case["ended"] and r % 8 == 5:
            parent = [-1] * case["W"]
        got.append((shared, tail, parent))
    return got


def _pages(n, page):
    return -(-n // page)


def _row_bytes(case):
    """Bytes of a row (a token and head of k or v) in the cache."""
    return case["d"] + 4 if case["code"] else 2 * case["d"]


def work(case):
    if case["op"] == "beam":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["R"] * case["W"] * case["V"]
        return {"bytes": size * n + 4 * case["R"] * case["W"] + 12 * case["R"] * case["K"], "flops": 3 * n}
    if case["op"] == "reorder":
        W, page = case["W"], case["page"]
        width = max(_pages(a + b, page) for a, b, _ in _beams(case)) + 1
        total = 8 * case["R"] * W * width + 12 * case["R"] * W
        for shared, tail, parent in _beams(case):
            kept = {p for p in parent if p >= 0}
            copies = len([p for p in parent if p >= 0]) - len(kept)
            total += 2 * copies * ((shared + tail) % page) * 2 * case["layers"] * case["Hk"] * _row_bytes(case)
            total += 4 * (W - len(kept)) * (_pages(shared + tail, page) - shared // page)
        return {"bytes": total, "flops": 0}
    ctx, new = _lengths(case)
    if case["op"] == "read":
        rows = 2 * sum(ctx) * case["Hk"]
        return {"bytes": rows * (_row_bytes(case) + 2 * case["d"]), "flops": rows * case["d"]}
    T = sum(new)
    if case["op"] == "store":
        kv = 2 * T * case["Hk"]  # read, written in 8 bits, and those read back
        return {"bytes": 4 * T * case["H"] * case["d"] + kv * (4 * case["d"] + 2 * _row_bytes(case)) + T * (8 + 4 * case["axes"]),
                "flops": 6 * T * (case["H"] + case["Hk"]) * case["pairs"] + 4 * kv * case["d"]}
    keys = sum(ctx) + T
    seen = sum(n * c + (n * (n + 1) // 2 if case["causal"] else n * n) for c, n in zip(ctx, new))
    return {"bytes": 2 * keys * case["Hk"] * _row_bytes(case) + 4 * T * case["H"] * case["d"],
            "flops": 4 * case["d"] * case["H"] * seen}


# ------------------------------------------------------------------ inputs


def _frequencies(case, dev):
    """inv_freq (float64) and axis (int32) of every pair; the axes share one falling sequence of frequencies."""
    P, A = case["pairs"], case["axes"]
    inv = [10000.0 ** -(i / P) for i in range(P)]
    axis = [i * A // P for i in range(P)]
    return torch.tensor(inv, dtype=torch.float64, device=dev), torch.tensor(axis, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    i32 = {"dtype": torch.int32, "device": dev}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def values(*shape):
        return normal(*shape).to(DTYPES[case["dtype"]])

    def cache(*shape):
        """One of a cache's two tensors and its scales (None: 16-bit values), as earlier steps left them."""
        if not case["code"]:
            return torch.stack([values(*shape[1:]) for _ in range(shape[0])]), None
        code, scale = torch.empty(shape, dtype=CODES[case["code"]], device=dev), torch.empty(shape[:-1], device=dev)
        for x, y in zip(code, scale):
            x.copy_((normal(*shape[1:]) * (TOP[case["code"]] / 3)).clamp_(-TOP[case["code"]], TOP[case["code"]]).round_())
            y.copy_((0.3 * normal(*shape[1:-1])).exp_() * (3 / TOP[case["code"]]))
        return code, scale

    def table(need, ids):
        """Block table of sequences of `need` pages each."""
        width = max(need) + 1
        held = torch.arange(width, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
        t = torch.full((len(need), width), -1, **i32)
        t[held] = ids[: sum(need)]
        return t

    s = {"op": case["op"], "case": case}
    if case["op"] == "beam":
        R, W, V = case["R"], case["W"], case["V"]
        s["logits"] = (3.0 * normal(R, W, V)).to(DTYPES[case["dtype"]])
        if case["masked"]:
            s["logits"].masked_fill_(torch.rand(V, generator=g, device=dev) < 0.2, -math.inf)
        s["scores"] = -10.0 * normal(R, W).abs()
        if case["dead"]:
            s["scores"][torch.rand((R, W), generator=g, device=dev) < 0.2] = -math.inf
        return s
    page, Hk, d = case["page"], case["Hk"], case["d"]
    if case["op"] == "reorder":
        W, beams = case["W"], _beams(case)
        order = torch.randperm(len(beams), generator=torch.Generator().manual_seed(seed)).tolist()
        beams = [beams[i] for i in order]
        need = [_pages(a + b, page) for a, b, _ in beams]
        first = [a // page for a, b, _ in beams]  # pages that a request's beams share
        private = [n - f for n, f in zip(need, first)]
        used = sum(first) + W * sum(private)
        total = used + W * len(beams) + 3
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        width = max(need) + 1
        t = torch.full((len(beams), W, width), -1, **i32)
        at = 0
        for r, (f, n) in enumerate(zip(first, private)):
            t[r, :, :f] = ids[at: at + f]
            t[r, :, f: f + n] = ids[at + f: at + f + W * n].reshape(W, n)
            at += f + W * n
        s["block_table"] = t.reshape(-1, width)
        s["lens"] = torch.tensor([a + b for a, b, _ in beams for _ in range(W)], **i32)
        s["parent"] = torch.tensor([p for _, _, p in beams], **i32)
        # the ring of free pages: those not held, from an odd place on
        free, head = total - used, 3 * total + total // 3
        s["ring"] = torch.full((total,), -1, **i32)
        s["ring"][(head + torch.arange(free, device=dev)) % total] = ids[used:]
        s["ring_state"] = torch.tensor([head, head + free], dtype=torch.int64, device=dev)
        (s["k"], s["ks"]), (s["v"], s["vs"]) = (cache(case["layers"], total, Hk, page, d) for _ in range(2))
        return s
    ctx, new = _lengths(case)
    order = torch.randperm(case["S"], generator=torch.Generator().manual_seed(seed)).tolist()
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    need = [_pages(c + n, page) for c, n in zip(ctx, new)]
    pages = sum(need) + 2
    s["block_table"] = table(need, torch.randperm(pages, generator=g, device=dev).to(torch.int32))
    (s["k_cache"], s["ks"]), (s["v_cache"], s["vs"]) = ((c[0], x[0]) for c, x in (cache(1, pages, Hk, page, d) for _ in range(2)))
    rows = ctx if case["op"] == "read" else new
    T = sum(rows)
    s["cu"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], **i32)
    s["kv_len"] = torch.tensor([c + n for c, n in zip(ctx, new)], **i32)
    s["tokens"] = T
    if case["op"] == "attn":
        s["q"] = values(T, case["H"], d)
        s["max_q"], s["max_kv"] = max(new), max(c + n for c, n in zip(ctx, new))
    if case["op"] == "store":
        s["inv_freq"], s["axis"] = _frequencies(case, dev)
        # keys of a channel or two that are far larger than the others, as models have them
        s["q"], s["k"], s["v"] = values(T, case["H"], d), values(T, Hk, d), values(T, Hk, d)
        s["k"][..., d // 3] *= 6
        s["start"] = torch.tensor(ctx, **i32)
        seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev), output_size=T)
        at = s["start"].long()[seq] + torch.arange(T, device=dev) - s["cu"].long()[seq]
        s["slots"] = s["block_table"].long()[seq, at // page] * page + at % page
        s["positions"] = torch.stack([at.int()] + [torch.randint(0, 1000, (T,), generator=g, **i32)] * (case["axes"] - 1), -1)
    return s


# -------------------------------------------------------------- plain forms


def _rotate(x, cos, sin, interleaved):
    """x [T, H, d] in 32 bits; cos, sin [T, 1, P]."""
    P = cos.shape[-1]
    if interleaved:
        x0, x1, rest = x[..., 0:2 * P:2], x[..., 1:2 * P:2], x[..., 2 * P:]
        y = torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2)
        return torch.cat((y, rest), -1)
    x0, x1, rest = x[..., :P], x[..., P:2 * P], x[..., 2 * P:]
    return torch.cat((x0 * cos - x1 * sin, x1 * cos + x0 * sin, rest), -1)


def _quantise(x, code):
    """Codes and scales of rows x [..., d] in 32 bits."""
    top = x.abs().amax(-1, keepdim=True)
    top = torch.where(top < TINY, 0.0, top)
    y = torch.where(top > 0, x * (TOP[code] / top), 0.0)
    y = y.round() if code == "int8" else y
    return y.clamp(-TOP[code], TOP[code]).to(CODES[code]), (top / TOP[code])[..., 0]


def _gather(s, cache, scale, start):
    """Cached rows [T, Hk, d] of the packed tokens, in 32 bits."""
    page = s["case"]["page"]
    t = torch.arange(s["tokens"], device=cache.device)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = (0 if start is None else start.long()[seq]) + t - cu[seq]
    where = (s["block_table"].long()[seq, at // page], slice(None), at % page)
    return cache.view(torch.int8)[where].view(cache.dtype).float() * scale[where][..., None]


def _plain_read(s, start=None):
    dtype = DTYPES[s["case"]["dtype"]]
    return {"k": _gather(s, s["k_cache"], s["ks"], start).to(dtype), "v": _gather(s, s["v_cache"], s["vs"], start).to(dtype)}


def _plain_store(s):
    c = s["case"]
    a = s["positions"][:, s["axis"].long()].double() * s["inv_freq"]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(s["q"].dtype)
    where = (s["slots"] // c["page"], slice(None), s["slots"] % c["page"])
    for x, cache, scale in ((_rotate(s["k"].float(), cos, sin, c["interleaved"]), "k_cache", "ks"), (s["v"].float(), "v_cache", "vs")):
        code, s[scale][where] = _quantise(x, c["code"])
        s[cache].view(torch.int8)[where] = code.view(torch.int8)
    return {"q": q} | _plain_read(s, s["start"])


def _plain_attn(s):
    c = s["case"]
    d, Hk, group, page = c["d"], c["Hk"], c["H"] // c["Hk"], c["page"]
    dev, T, L, Q = s["q"].device, s["q"].shape[0], s["max_kv"], s["max_q"]
    cu, kv = s["cu"].long(), s["kv_len"].long()
    S = kv.numel()
    new = cu[1:] - cu[:-1]
    key = torch.arange(L, device=dev)
    held = key[None] < kv[:, None]
    at = (s["block_table"].long()[:, key // page].clamp(min=0), slice(None), (key % page)[None])

    def read(cache, scale):
        return (cache.view(torch.int8)[at].view(cache.dtype).float() * scale[at][..., None]).permute(0, 2, 1, 3)

    j = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + j[None]).clamp(max=T - 1)
    q = s["q"][row].float().reshape(S, Q, Hk, group, d).permute(0, 2, 3, 1, 4).reshape(S, Hk, group * Q, d)
    x = q @ read(s["k_cache"], s["ks"]).transpose(-1, -2) * (1.0 / math.sqrt(d))
    del q
    if c["causal"]:
        last = (kv - new)[:, None] + j[None]
        see = key[None, None] <= torch.minimum(last, kv[:, None] - 1)[:, :, None]
    else:
        see = held[:, None].expand(S, Q, L)
    x = x.reshape(S, Hk, group, Q, L).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = torch.where(held[:, None, :, None], read(s["v_cache"], s["vs"]), 0.0)
    o = (p.reshape(S, Hk, group * Q, L) @ v).reshape(S, Hk, group, Q, d)
    o = torch.where(l > 0, o / l, 0.0)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(S, Q, c["H"], d)[seq, t - cu[seq]].to(s["q"].dtype)}


def _plain_beam(s):
    x, K, V = s["logits"].double(), s["case"]["K"], s["case"]["V"]
    m = x.amax(-1, keepdim=True)
    lse = m + (x - m).exp().sum(-1, keepdim=True).log()
    x = (s["scores"].double()[..., None] + (x - lse)).flatten(1)
    x = torch.where(x.abs() < math.inf, x, -math.inf)  # (what is not a number is no candidate)
    best, at = torch.sort(x, dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    if best.shape[1] < K:
        more = (0, K - best.shape[1])
        best, at = torch.nn.functional.pad(best, more, value=-math.inf), torch.nn.functional.pad(at, more)
    none = best == -math.inf
    return {"scores": best.float(), "parent": torch.where(none, -1, at // V).int(), "token": torch.where(none, -1, at % V).int()}


def _plain_reorder(s):
    W, page, ring = s["case"]["W"], s["case"]["page"], s["ring"]
    R, F, dev = s["parent"].shape[0], ring.numel(), ring.device
    table = s["block_table"].reshape(R, W, -1).long()
    lens, parent = s["lens"].reshape(R, W).long(), s["parent"].long()
    head, tail = s["ring_state"][0], s["ring_state"][1]
    w = torch.arange(W, device=dev)
    before = w[None] < w[:, None]

    def again(p):  # an earlier beam continues the same one, and its last page is not full
        twice = ((p[:, :, None] == p[:, None]) & before).any(-1) & (p >= 0)
        return twice & (lens.gather(1, p.clamp(min=0)) % page != 0)

    need = again(parent).sum(1)
    done = (need.cumsum(0) <= tail - head) | (need == 0)
    parent = torch.where(done[:, None], parent, w[None])
    copied = again(parent) & done[:, None]
    src, live = parent.clamp(min=0), parent >= 0
    out_lens = torch.where(live, lens.gather(1, src), 0)
    pages = (out_lens + page - 1) // page
    col = torch.arange(table.shape[2], device=dev)
    out = table.gather(1, src[:, :, None].expand_as(table))
    out = torch.where(col < pages[:, :, None], out, -1)
    i, j = torch.nonzero(copied, as_tuple=True)
    last = pages[i, j] - 1
    old, fresh = out[i, j, last], ring[(head + torch.arange(i.numel(), device=dev)) % F].long()
    out[i, j, last] = fresh
    # pages that no beam holds any more go back, in the order of requests, columns and beams
    held = col < ((lens + page - 1) // page)[:, :, None]
    kept = (parent[:, :, None] == w).any(1) & done[:, None]
    kept = kept | ~done[:, None]
    same = (table[:, :, None] == table[:, None]) & held[:, :, None] & held[:, None]
    stays = (same & kept[:, None, :, None]).any(2)
    other = (same & before[None, :, :, None]).any(2)
    back = (held & ~stays & ~other).permute(0, 2, 1)
    gone = table.permute(0, 2, 1)[back]
    ring[(tail + torch.arange(gone.numel(), device=dev)) % F] = gone.int()
    # rows of the last pages that beams continue separately
    rows = out_lens[i, j] % page
    n, r = torch.nonzero(torch.arange(page, device=dev)[None] < rows[:, None], as_tuple=True)
    for x in (s["k"], s["v"], s["ks"], s["vs"]):
        if x is not None:
            y = x.view(torch.int8) if x.element_size() == 1 else x
            y[:, fresh[n], :, r] = y[:, old[n], :, r]
    state = torch.stack((head + i.numel(), tail + gone.numel()))
    return {"block_table": out.reshape(R * W, -1).int(), "lens": out_lens.reshape(-1).int(), "ring_state": state, "done": done.int(),
            "ring": ring} | _values(s)


def _values(s):
    """The caches' contents as the values they stand for: the codes as numbers, and the scales."""
    if not s["case"]["code"]:
        return {"k": s["k"], "v": s["v"]}
    code = {"k": s["k"], "v": s["v"]} if s["case"]["code"] == "e4m3" else {"k": s["k"].view(torch.int8), "v": s["v"].view(torch.int8)}
    return code | {"ks": s["ks"], "vs": s["vs"]}


# ---------------------------------------------------- the framework's calls


def _own_read(s, start=None):
    from certified_fixed_stabilizer_gb300 import clis
    k, v = clis.paged_read(s["k_cache"], s["v_cache"], s["block_table"], s["cu"], s["tokens"], start=start, k_scale=s["ks"],
                           v_scale=s["vs"], dtype=DTYPES[s["case"]["dtype"]])
    return {"k": k, "v": v}


def _own_store(s):
    from certified_fixed_stabilizer_gb300 import clis
    q = clis.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"], positions=s["positions"],
                          inv_freq=s["inv_freq"], axis=s["axis"], interleaved=s["case"]["interleaved"], k_scale=s["ks"], v_scale=s["vs"])
    return {"q": q} | _own_read(s, s["start"])


def _own_attn(s):
    from certified_fixed_stabilizer_gb300 import clis
    return {"o": clis.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu"], s["kv_len"], s["max_q"],
                                      causal=s["case"]["causal"], k_scale=s["ks"], v_scale=s["vs"])}


def _own_beam(s):
    from certified_fixed_stabilizer_gb300 import clis
    b = clis.beam_select(s["logits"], s["scores"], s["case"]["K"])
    return {"scores": b.scores, "parent": b.parent, "token": b.token}


def _own_reorder(s):
    from certified_fixed_stabilizer_gb300 import clis
    r = clis.paged_reorder(s["lens"], s["parent"], s["block_table"], s["ring"], s["ring_state"],
                           [x for x in (s["k"], s["v"]) if x is not None], [x for x in (s["ks"], s["vs"]) if x is not None])
    return {"block_table": r.block_table, "lens": r.lens, "ring_state": r.ring_state, "done": r.done, "ring": s["ring"]} | _values(s)


def run(state):
    if own:
        return {"store": _own_store, "read": _own_read, "attn": _own_attn, "beam": _own_beam, "reorder": _own_reorder}[state["op"]](state)
    return {"store": _plain_store, "read": _plain_read, "attn": _plain_attn, "beam": _plain_beam, "reorder": _plain_reorder}[state["op"]](state)


# -------------------------------------------------- the definitions in 64 bits


def _turn(x, positions, inv_freq, axis, interleaved):
    """The rotation as a product of complex numbers, in 64 bits: x [T, H, d], positions [T, A]."""
    x, P = x.double(), inv_freq.numel()
    a = (positions.double().index_select(-1, axis.long()) * inv_freq)[:, None]
    turn = torch.polar(torch.ones_like(a), a)
    if interleaved:
        z = torch.view_as_complex(x[..., : 2 * P].reshape(*x.shape[:-1], P, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * P)
    else:
        z = torch.complex(x[..., :P].contiguous(), x[..., P:2 * P].contiguous()) * turn
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., 2 * P:]), -1)


def _held(x, code):
    """What a cache of 8 bits holds of the rows x, in 64 bits."""
    unit = x.abs().max(-1, keepdim=True).values / TOP[code]
    y = x / torch.where(unit > 0, unit, 1.0)
    step = 1.0 if code == "int8" else torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * unit


def exact(case, seed):
    if case["op"] == "reorder":
        return None
    s = prepare(case, seed)
    if case["op"] == "beam":
        lse = torch.logsumexp(s["logits"].double(), -1, keepdim=True)
        x = (s["logits"].double() - lse + s["scores"].double()[..., None]).flatten(1)
        x[~torch.isfinite(x)] = -math.inf
        K = min(case["K"], x.shape[1])
        best = torch.topk(x, K, -1).values
        return {"scores": torch.cat((best, torch.full((case["R"], case["K"] - K), -math.inf, dtype=best.dtype, device=best.device)), 1),
                "parent": None, "token": None}
    page, Hk, d = case["page"], case["Hk"], case["d"]
    if case["op"] == "store":
        f = (s["positions"], s["inv_freq"], s["axis"], case["interleaved"])
        return {"q": _turn(s["q"], *f), "k": _held(_turn(s["k"], *f), case["code"]), "v": _held(s["v"].double(), case["code"])}

    def rows(cache, scale, i, n):
        pages = s["block_table"][i, : _pages(n, page)].long()
        x = cache.view(torch.int8)[pages].view(cache.dtype).float().double() * scale[pages].double()[..., None]
        return x.transpose(0, 1).reshape(Hk, -1, d)[:, :n]

    cu, kv = s["cu"].tolist(), s["kv_len"].tolist()
    if case["op"] == "read":
        return {"k": torch.cat([rows(s["k_cache"], s["ks"], i, n).transpose(0, 1) for i, n in enumerate(kv)]),
                "v": torch.cat([rows(s["v_cache"], s["vs"], i, n).transpose(0, 1) for i, n in enumerate(kv)])}
    group = case["H"] // Hk
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(kv):
        a, b = cu[i], cu[i + 1]
        k, v = rows(s["k_cache"], s["ks"], i, n), rows(s["v_cache"], s["vs"], i, n)
        late = torch.arange(n, device=o.device)[None] > torch.arange(n - (b - a), n, device=o.device)[:, None]
        for h in range(case["H"]):
            x = s["q"][a:b, h].double() @ k[h // group].t() / math.sqrt(d)
            if case["causal"]:
                x = x.masked_fill(late, -math.inf)
            o[a:b, h] = torch.softmax(x, -1) @ v[h // group]
    return {"o": o}
