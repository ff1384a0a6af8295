"""What is measured of the operators around a key/value cache: rotary positions with several axes, the plan of a
serving step (block tables and slots), the write of new keys and values into a paged cache, and attention of new
tokens over that cache.  ``run`` computes each in elementary torch operations, or, with ``own``, through
``certified_fixed_stabilizer_gb300.clis``.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # q and k of one layer of 480p video attention (20 heads, a 21 x 30 x 52 token grid), (time, height, width) axes.
        {"name": "rope_video", "op": "rope", "B": 1, "H": 20, "Hk": 20, "grid": "21x30x52", "N": 32760, "d": 128,
         "pairs": 64, "axes": 3, "shared": False, "interleaved": True, "far": 1, "grad": False, "dtype": "bf16"},
        # A training step's q and k with shared key heads: text far into a document among image tokens; y and gradients.
        {"name": "rope_train", "op": "rope", "B": 2, "H": 32, "Hk": 8, "grid": "", "N": 4099, "d": 128,
         "pairs": 64, "axes": 3, "shared": True, "interleaved": False, "far": 1000000, "grad": True, "dtype": "fp16"},
        # A few tokens with a quarter of each head rotated, one axis: latency alone.
        {"name": "rope_few", "op": "rope", "B": 1, "H": 16, "Hk": 2, "grid": "", "N": 7, "d": 64,
         "pairs": 8, "axes": 1, "shared": True, "interleaved": False, "far": 32000, "grad": False, "dtype": "bf16"},
        # One decoding step of 8 requests.
        {"name": "plan_few", "op": "plan", "S": 8, "page": 16, "ctx": 4000, "new": 1, "chunks": 0, "lens": 1},
        # A large batch: a thousand requests, some of them long prompts, some finished.
        {"name": "plan_many", "op": "plan", "S": 1024, "page": 16, "ctx": 8000, "new": 2048, "chunks": 100, "lens": 2},
        # New keys and values of 64 decoding requests, rotated and written.
        {"name": "append_decode", "op": "append", "T": 64, "H": 32, "Hk": 8, "d": 128, "page": 16, "pairs": 64,
         "axes": 1, "interleaved": False, "far": 30000, "dtype": "bf16"},
        # A prompt's chunk with video positions.
        {"name": "append_chunk", "op": "append", "T": 8192, "H": 32, "Hk": 8, "d": 128, "page": 64, "pairs": 64,
         "axes": 3, "interleaved": True, "far": 100000, "dtype": "fp16"},
        # One request, a short cache: latency alone.
        {"name": "attn_one", "op": "attn", "S": 1, "new": 1, "chunks": 0, "ctx": 300, "even": True, "H": 32, "Hk": 8,
         "d": 128, "page": 16, "causal": True, "dtype": "bf16", "lens": 3},
        # Single tokens of 64 requests of very different lengths: the cache's bytes.
        {"name": "attn_decode", "op": "attn", "S": 64, "new": 1, "chunks": 0, "ctx": 16000, "even": False, "H": 32,
         "Hk": 8, "d": 128, "page": 16, "causal": True, "dtype": "bf16", "lens": 4},
        # Drafted tokens (up to 5 a request) over a cache of 64-wide heads.
        {"name": "attn_draft", "op": "attn", "S": 17, "new": 5, "chunks": 17, "ctx": 9001, "even": False, "H": 16,
         "Hk": 4, "d": 64, "page": 64, "causal": True, "dtype": "fp16", "lens": 5},
        # A chunk of a long prompt behind 30,000 cached tokens: the tensor cores.
        {"name": "attn_chunk", "op": "attn", "S": 1, "new": 2048, "chunks": 1, "ctx": 30011, "even": True, "H": 32,
         "Hk": 8, "d": 128, "page": 64, "causal": True, "dtype": "bf16", "lens": 6},
        # A serving step of both: three prompts' chunks among decoding requests.
        {"name": "attn_mixed", "op": "attn", "S": 12, "new": 513, "chunks": 3, "ctx": 8000, "even": False, "H": 32,
         "Hk": 8, "d": 128, "page": 32, "causal": True, "dtype": "bf16", "lens": 7},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "append", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "plan":
        S = _log(rng, 1, 1024)
        return {"op": "plan", "S": S, "page": rng.choice([8, 16, 32, 64, 128]), "ctx": _log(rng, 1, 8000),
                "new": _log(rng, 1, 2048), "chunks": rng.randint(0, min(S, 100)), "lens": rng.randrange(1 << 20)}
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 3, 4, 5, 8])
    axes = rng.choice([1, 2, 3, 4])
    pairs = rng.choice([p for p in (8, 16, 24, 32, 48, 64) if p <= d // 2 and p >= axes])
    if op == "rope":
        return {"op": "rope", "B": rng.choice([1, 2, 3]), "H": H, "Hk": Hk, "grid": "", "N": _log(rng, 1, 8000), "d": d,
                "pairs": pairs, "axes": axes, "shared": rng.random() < 0.5, "interleaved": rng.random() < 0.5,
                "far": _log(rng, 100, 4000000), "grad": rng.random() < 0.5, "dtype": dtype}
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "append":
        return {"op": "append", "T": _log(rng, 1, 8192), "H": H, "Hk": Hk, "d": d, "page": page, "pairs": pairs,
                "axes": axes, "interleaved": rng.random() < 0.5, "far": _log(rng, 100, 4000000), "dtype": dtype}
    # attention: single and drafted tokens over many caches, or chunks; rows times keys stay under the listed ones'.
    if rng.random() < 0.5:
        S, new = _log(rng, 1, 64), _log(rng, 1, 8)
        ctx, chunks = _log(rng, 1, 16000), rng.randint(0, S)
    else:
        S, new = rng.randint(1, 6), _log(rng, 9, 1024)
        ctx, chunks = _log(rng, 1, 8000), rng.randint(1, S)
    return {"op": "attn", "S": S, "new": new, "chunks": chunks, "ctx": ctx, "even": rng.random() < 0.3, "H": H, "Hk": Hk,
            "d": d, "page": page, "causal": rng.random() < 0.8, "dtype": dtype, "lens": rng.randrange(1 << 20)}


def _lengths(case):
    """(cached, new) lengths of a case's sequences; a plan also has finished ones (new = -1)."""
    rng = random.Random(case["lens"])
    ctx, new = [], []
    for s in range(case["S"]):
        ctx.append(case["ctx"] if case.get("even") else rng.randint(case["ctx"] // 16, case["ctx"]))
        new.append(1 if s >= case["chunks"] else case["new"] if s == 0 else rng.randint(1, case["new"]))
    if case["op"] == "plan":
        new = [-1 if s % 16 == 9 else n for s, n in enumerate(new)]
    return ctx, new


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] == "rope":
        rows = case["B"] * (case["H"] + case["Hk"]) * case["N"]
        once = {"bytes": 2 * rows * case["d"] * 2 + 4 * case["B"] * case["N"] * case["axes"],
                "flops": 6 * rows * case["pairs"]}
        return {k: v * (2 if case["grad"] else 1) for k, v in once.items()}
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        page = case["page"]
        tokens = sum(max(n, 0) for n in new)
        taken = sum(_pages(c + max(n, 0), page) - _pages(c, page) for c, n in zip(ctx, new))
        back = sum(_pages(c, page) for c, n in zip(ctx, new) if n < 0)
        return {"bytes": 16 * case["S"] + 12 * tokens + 8 * taken + 8 * back, "flops": 0}
    if case["op"] == "append":
        rows = case["T"] * (case["H"] + 2 * case["Hk"])
        return {"bytes": 2 * rows * case["d"] * 2 + case["T"] * (8 + 4 * case["axes"]),
                "flops": 6 * case["T"] * (case["H"] + case["Hk"]) * case["pairs"]}
    ctx, new = _lengths(case)
    keys = sum(c + n for c, n in zip(ctx, new))
    seen = sum(n * c + (n * (n + 1) // 2 if case["causal"] else n * n) for c, n in zip(ctx, new))
    return {"bytes": 4 * keys * case["Hk"] * case["d"] + 4 * sum(new) * case["H"] * case["d"] + 4 * sum(new) * case["H"],
            "flops": 4 * case["d"] * case["H"] * seen}


# ------------------------------------------------------------------ inputs


def _frequencies(case, dev):
    """inv_freq (float64) and axis (int32) of every pair: the axes share one falling sequence of frequencies, or each
    has its own, as for the blocks of a video token's position."""
    P, A = case["pairs"], case["axes"]
    size = [P - (A - 1) * (P // A)] + [P // A] * (A - 1)
    axis = [a for a in range(A) for _ in range(size[a])]
    place = [i / P for i in range(P)] if case.get("shared", True) else [i / n for n in size for i in range(n)]
    inv = [10000.0 ** -x for x in place]
    return torch.tensor(inv, dtype=torch.float64, device=dev), torch.tensor(axis, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(DTYPES[case["dtype"]])

    def whole(hi, *shape):
        return torch.randint(0, hi, shape, generator=g, device=dev, dtype=torch.int32)

    s = {"op": case["op"], "case": case}
    if case["op"] in ("rope", "append"):
        s["inv_freq"], s["axis"] = _frequencies(case, dev)
    if case["op"] == "rope":
        B, N, A = case["B"], case["N"], case["axes"]
        s["q"], s["k"] = normal(B, case["H"], N, case["d"]), normal(B, case["Hk"], N, case["d"])
        if case["grid"]:
            sides = [int(x) for x in case["grid"].split("x")]
            at = [torch.arange(n, dtype=torch.int32, device=dev) for n in sides]
            s["positions"] = torch.stack(torch.meshgrid(*at, indexing="ij"), -1).reshape(1, N, A).contiguous()
        else:
            s["positions"] = whole(case["far"], B, N, A)
        if case["grad"]:
            s["gq"], s["gk"] = normal(B, case["H"], N, case["d"]), normal(B, case["Hk"], N, case["d"])
        return s
    if case["op"] == "append":
        T, page = case["T"], case["page"]
        pages = _pages(T, page) * 2 + 3
        s["q"], s["k"], s["v"] = normal(T, case["H"], case["d"]), normal(T, case["Hk"], case["d"]), normal(T, case["Hk"], case["d"])
        s["k_cache"], s["v_cache"] = normal(pages, case["Hk"], page, case["d"]), normal(pages, case["Hk"], page, case["d"])
        # runs of neighbouring slots, as a request's chunk has, and a padding row
        runs = torch.randperm(pages * page // 8, generator=g, device=dev)[: _pages(T, 8)]
        s["slots"] = (8 * runs[:, None] + torch.arange(8, device=dev)).reshape(-1)[:T].contiguous()
        if T > 8:
            s["slots"][-1] = -1
        s["positions"] = whole(case["far"], 1, T, case["axes"])
        return s
    ctx, new = _lengths(case)
    S, page = case["S"], case["page"]
    order = torch.randperm(S, generator=torch.Generator().manual_seed(seed)).tolist()
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    have = [_pages(c, page) for c in ctx]
    need = [_pages(c + max(n, 0), page) for c, n in zip(ctx, new)]
    width = max(need) + 1
    i32 = {"dtype": torch.int32, "device": dev}
    if case["op"] == "plan":
        total = sum(need) + 5
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        held = torch.arange(width, device=dev)[None] < torch.tensor(have, device=dev)[:, None]
        s["block_table"] = torch.full((S, width), -1, **i32)
        s["block_table"][held] = ids[: sum(have)]
        # the ring of free pages: those not held, from an odd place on
        free = total - sum(have)
        head = 3 * total + total // 3
        s["ring"] = torch.full((total,), -1, **i32)
        s["ring"][(head + torch.arange(free, device=dev)) % total] = ids[sum(have):]
        s["ring_state"] = torch.tensor([head, head + free], dtype=torch.int64, device=dev)
        s["ctx_len"], s["new_len"] = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
        s["tokens"] = sum(max(n, 0) for n in new)
        return s
    T = sum(new)
    pages = sum(need) + 2
    s["q"] = normal(T, case["H"], case["d"])
    s["k_cache"], s["v_cache"] = normal(pages, case["Hk"], page, case["d"]), normal(pages, case["Hk"], page, case["d"])
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    held = torch.arange(width, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    s["block_table"] = torch.full((S, width), -1, **i32)
    s["block_table"][held] = ids[: sum(need)]
    s["cu_q"] = torch.tensor([sum(new[:i]) for i in range(S + 1)], **i32)
    s["kv_len"] = torch.tensor([c + n for c, n in zip(ctx, new)], **i32)
    s["max_q"], s["max_kv"] = max(new), max(c + n for c, n in zip(ctx, new))
    return s


# -------------------------------------------------------------- plain forms


def _angles(positions, inv_freq, axis):
    """cos and sin [B, N, P] in 32 bits; the angles themselves in 64 (positions reach millions)."""
    a = positions[..., axis.long()].double() * inv_freq
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, interleaved):
    """x [..., N, d] in 32 bits; cos, sin broadcast against [..., N, P]."""
    P = cos.shape[-1]
    if interleaved:
        x0, x1, rest = x[..., 0:2 * P:2], x[..., 1:2 * P:2], x[..., 2 * P:]
        y = torch.stack((x0 * cos - x1 * sin, x1 * cos + x0 * sin), -1).flatten(-2)
        return torch.cat((y, rest), -1)
    x0, x1, rest = x[..., :P], x[..., P:2 * P], x[..., 2 * P:]
    return torch.cat((x0 * cos - x1 * sin, x1 * cos + x0 * sin, rest), -1)


def _plain_rope(s):
    inter = s["case"]["interleaved"]
    cos, sin = (t[:, None] for t in _angles(s["positions"], s["inv_freq"], s["axis"]))
    out = {"q": _rotate(s["q"].float(), cos, sin, inter).to(s["q"].dtype),
           "k": _rotate(s["k"].float(), cos, sin, inter).to(s["k"].dtype)}
    if "gq" in s:
        out["dq"] = _rotate(s["gq"].float(), cos, -sin, inter).to(s["q"].dtype)
        out["dk"] = _rotate(s["gk"].float(), cos, -sin, inter).to(s["k"].dtype)
    return out


def _plain_append(s):
    page = s["case"]["page"]
    cos, sin = (t[0][:, None] for t in _angles(s["positions"], s["inv_freq"], s["axis"]))
    q = _rotate(s["q"].float(), cos, sin, s["case"]["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, s["case"]["interleaved"]).to(s["k"].dtype)
    row = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][row]
    s["k_cache"][at // page, :, at % page] = k[row]
    s["v_cache"][at // page, :, at % page] = s["v"][row]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_plan(s):
    ctx, page, ring = s["ctx_len"].long(), s["case"]["page"], s["ring"]
    new, gone = s["new_len"].long().clamp(min=0), s["new_len"] < 0
    dev, S, width, F = ctx.device, ctx.numel(), s["block_table"].shape[1], ring.numel()
    total = torch.where(gone, torch.zeros_like(ctx), ctx + new)
    have = (ctx + page - 1) // page
    need = torch.where(gone, have, (total + page - 1) // page)
    taken, back = need - have, torch.where(gone, have, torch.zeros_like(have))
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    first = taken.cumsum(0) - taken
    head, tail = s["ring_state"][0], s["ring_state"][1]
    col = torch.arange(width, device=dev)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    page_of = ring[(head + first[:, None] + col - have[:, None]) % F]
    s["block_table"].copy_(torch.where(fresh, page_of, s["block_table"]))
    given = gone[:, None] & (col < have[:, None])
    place = (tail + (back.cumsum(0) - back)[:, None] + col) % F
    ring[place[given]] = s["block_table"][given]
    t = torch.arange(s["tokens"], device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[seq] + t - cu[seq]
    slots = s["block_table"][seq, pos // page].long() * page + pos % page
    return {"cu_q": cu.int(), "kv_len": total.int(), "slots": slots, "positions": pos.int(),
            "ring_state": torch.stack((head + taken.sum(), tail + back.sum())), "block_table": s["block_table"], "ring": ring}


def _plain_attn(s):
    c = s["case"]
    d, Hk, group, page = c["d"], c["Hk"], c["H"] // c["Hk"], c["page"]
    dev, T, L, Q = s["q"].device, s["q"].shape[0], s["max_kv"], s["max_q"]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    S = kv.numel()
    new = cu[1:] - cu[:-1]
    key = torch.arange(L, device=dev)
    held = key[None] < kv[:, None]
    at = s["block_table"].long()[:, key // page].clamp(min=0)
    k = s["k_cache"][at, :, (key % page)[None]].float().permute(0, 2, 1, 3)
    v = torch.where(held[:, :, None, None], s["v_cache"][at, :, (key % page)[None]].float(), 0.0).permute(0, 2, 1, 3)
    j = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + j[None]).clamp(max=T - 1)
    q = s["q"][row].float().reshape(S, Q, Hk, group, d).permute(0, 2, 3, 1, 4).reshape(S, Hk, group * Q, d)
    x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    del k, q
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
    o = (p.reshape(S, Hk, group * Q, L) @ v).reshape(S, Hk, group, Q, d)
    o = torch.where(l > 0, o / l, 0.0)
    lse2 = (m + l.log())[..., 0] * math.log2(math.e)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    o = o.permute(0, 3, 1, 2, 4).reshape(S, Q, c["H"], d)[seq, t - cu[seq]]
    lse2 = lse2.permute(0, 3, 1, 2).reshape(S, Q, c["H"])[seq, t - cu[seq]]
    return {"o": o.to(s["q"].dtype), "lse2": lse2}


# ---------------------------------------------------- the framework's calls


def _own_rope(s):
    from certified_fixed_stabilizer_gb300 import clis
    args = (s["positions"], s["inv_freq"], s["axis"])
    inter = s["case"]["interleaved"]
    if "gq" not in s:
        q, k = clis.rope(s["q"], s["k"], *args, interleaved=inter)
        return {"q": q, "k": k}
    q0, k0 = s["q"].detach().requires_grad_(), s["k"].detach().requires_grad_()
    q, k = clis.rope_autograd(q0, k0, *args, interleaved=inter)
    dq, dk = torch.autograd.grad((q, k), (q0, k0), (s["gq"], s["gk"]))
    return {"q": q, "k": k, "dq": dq, "dk": dk}


def _own_append(s):
    from certified_fixed_stabilizer_gb300 import clis
    q = clis.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"], positions=s["positions"][0],
                          inv_freq=s["inv_freq"], axis=s["axis"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_plan(s):
    from certified_fixed_stabilizer_gb300 import clis
    p = clis.paged_plan(s["ctx_len"], s["new_len"], s["block_table"], s["ring"], s["ring_state"], s["case"]["page"], s["tokens"])
    return {"cu_q": p.cu_q, "kv_len": p.kv_len, "slots": p.slots, "positions": p.positions, "ring_state": p.ring_state,
            "block_table": s["block_table"], "ring": s["ring"]}


def _own_attn(s):
    from certified_fixed_stabilizer_gb300 import clis
    o, lse2 = clis.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"], s["kv_len"], s["max_q"],
                                   causal=s["case"]["causal"], return_lse=True)
    return {"o": o, "lse2": lse2}


def run(state):
    if own:
        return {"rope": _own_rope, "append": _own_append, "plan": _own_plan, "attn": _own_attn}[state["op"]](state)
    return {"rope": _plain_rope, "append": _plain_append, "plan": _plain_plan, "attn": _plain_attn}[state["op"]](state)


# -------------------------------------------------- the definitions in 64 bits


def _turn(x, positions, inv_freq, axis, interleaved, sign=1.0):
    """The rotation as a product of complex numbers, in 64 bits: x [..., N, d], positions [N, A] (or [B, 1, N, A])."""
    x, P = x.double(), inv_freq.numel()
    a = sign * positions.double().index_select(-1, axis.long()) * inv_freq
    turn = torch.polar(torch.ones_like(a), a)
    if interleaved:
        z = torch.view_as_complex(x[..., : 2 * P].reshape(*x.shape[:-1], P, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * P)
    else:
        z = torch.complex(x[..., :P].contiguous(), x[..., P:2 * P].contiguous()) * turn
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., 2 * P:]), -1)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        f = (s["positions"][:, None], s["inv_freq"], s["axis"], case["interleaved"])
        out = {"q": _turn(s["q"], *f), "k": _turn(s["k"], *f)}
        if case["grad"]:
            out |= {"dq": _turn(s["gq"], *f, -1.0), "dk": _turn(s["gk"], *f, -1.0)}
        return out
    if case["op"] == "append":
        f = (s["positions"][0][:, None], s["inv_freq"], s["axis"], case["interleaved"])
        q, k = _turn(s["q"], *f), _turn(s["k"], *f)
        kc, vc = s["k_cache"].double().transpose(1, 2), s["v_cache"].double().transpose(1, 2)
        kc, vc = kc.reshape(-1, *kc.shape[2:]), vc.reshape(-1, *vc.shape[2:])
        for t, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                kc[at], vc[at] = k[t], s["v"][t].double()
        back = (-1, case["page"], case["Hk"], case["d"])
        return {"q": q, "k_cache": kc.reshape(back).transpose(1, 2), "v_cache": vc.reshape(back).transpose(1, 2)}
    d, group, page = case["d"], case["H"] // case["Hk"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse2 = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device=o.device)
    cu, kv = s["cu_q"].tolist(), s["kv_len"].tolist()
    for i, n in enumerate(kv):
        a, b = cu[i], cu[i + 1]
        pages = s["block_table"][i, : _pages(n, page)].long()
        k = s["k_cache"][pages].transpose(0, 1).reshape(case["Hk"], -1, d)[:, :n]
        v = s["v_cache"][pages].transpose(0, 1).reshape(case["Hk"], -1, d)[:, :n]
        for h in range(case["H"]):
            x = s["q"][a:b, h].double() @ k[h // group].double().t() / math.sqrt(d)
            if case["causal"]:
                late = torch.arange(n, device=o.device)[None] > torch.arange(n - (b - a), n, device=o.device)[:, None]
                x = x.masked_fill(late, -math.inf)
            o[a:b, h] = torch.softmax(x, -1) @ v[h // group].double()
            lse2[a:b, h] = torch.logsumexp(x, -1) / math.log(2.0)
    return {"o": o, "lse2": lse2}
