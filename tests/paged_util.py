"""Inputs and 64-bit references for the tests around a paged cache (no method code)."""
import math
import random

import torch

# Half a step of each type, relative: a rounding is off by at most this.
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make_batch(ctx, new, H, Hkv, d, page, dtype, seed=0, device="cuda", extra_rows=0, spare=3, poison=True, layout="hnd"):
    """Random batch over a paged cache.  Pages are scattered; with ``poison`` every cache
    row that holds no key is NaN or inf and unused block-table entries are out of range."""
    g = torch.Generator(device=device).manual_seed(seed)
    rng = random.Random(seed)
    S = len(ctx)
    kv = [c + n for c, n in zip(ctx, new)]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    width = max(need + [0]) + 2
    bt = torch.full((S, width), 0x3FFFFFFF if poison else -1, dtype=torch.int32)
    shape = (pages, Hkv, page, d) if layout == "hnd" else (pages, page, Hkv, d)
    bad = float("nan") if seed % 2 else float("inf")
    kc, vc = (torch.full(shape, bad if poison else 0.0, dtype=dtype, device=device) for _ in range(2))
    if layout != "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    keys, vals, at = [], [], 0
    for s in range(S):
        mine = ids[at:at + need[s]]
        at += need[s]
        bt[s, :need[s]] = torch.tensor(mine, dtype=torch.int32)
        k, v = (torch.randn((kv[s], Hkv, d), generator=g, device=device).to(dtype) for _ in range(2))
        keys.append(k)
        vals.append(v)
        for i, p in enumerate(mine):
            n = min(page, kv[s] - i * page)
            kc[p, :, :n] = k[i * page:i * page + n].transpose(0, 1)
            vc[p, :, :n] = v[i * page:i * page + n].transpose(0, 1)
    T = sum(new) + extra_rows
    q = torch.randn((T, H, d), generator=g, device=device).to(dtype)
    cu = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device=device)
    return {"q": q, "k_cache": kc, "v_cache": vc, "block_table": bt.to(device), "cu_q": cu,
            "kv_len": torch.tensor(kv, dtype=torch.int32, device=device), "keys": keys, "vals": vals,
            "ctx": ctx, "new": new, "max_q": max(new + [1])}


def reference(b, scale=None, causal=True):
    """(o, lse2, |v| mean, sum of exp relative to the maximum, seen |v|) per row [T', H, ...] in 64 bits;
    T' = the rows that belong to sequences."""
    q = b["q"]
    H, d = q.shape[1:]
    Hkv = b["k_cache"].shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    outs = []
    for s, (c, n) in enumerate(zip(b["ctx"], b["new"])):
        if n == 0:
            continue
        r0 = sum(b["new"][:s])
        qs = q[r0:r0 + n].double().transpose(0, 1)                                  # [H, n, d]
        k = b["keys"][s].double().transpose(0, 1).repeat_interleave(H // Hkv, 0)
        v = b["vals"][s].double().transpose(0, 1).repeat_interleave(H // Hkv, 0)    # [H, kv, d]
        kv = c + n
        x = qs @ k.transpose(1, 2) * scale
        if causal:
            hide = torch.arange(kv, device=q.device)[None] > torch.arange(c, c + n, device=q.device)[:, None]
            x = x.masked_fill(hide, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        L = p.sum(-1, keepdim=True)
        o = p @ v / L
        A = p @ v.abs() / L
        seen = (p > 0).double() @ v.abs() / L
        lse2 = (m + L.log())[..., 0] / math.log(2.0)
        outs.append(tuple(t.transpose(0, 1) for t in (o, lse2, A, seen)))
    return tuple(torch.cat(t) for t in zip(*outs))


def check_attention(got_o, got_lse2, b, causal=True, scale=None, what=""):
    """Element-wise bounds derived from the arithmetic:
    * the output is rounded once (half a step of |o|);
    * every weight p is rounded once to the data type before it multiplies v: half a step of
      sum p |v| / sum p =: A; in fp16 weights below 2^-14 of the shift also lose up to 2^-25 each;
    * a score is a 32-bit dot product of d products of 16-bit values (exact): off by at most
      d 2^-24 sum |q k| scale; for unit normals sum |q k| is about 0.64 d, so x is off by at most
      128 * 2^-24 * 82 * 0.0884 = 5.5e-5 in the exponent, which moves o by at most twice that times A
      (numerator and denominator); exp2 and the 32-bit sums add some 1e-6.  2e-4 A covers them."""
    rows = got_o.shape[0]
    o, lse2, A, seen = reference(b, scale, causal)
    assert o.shape[0] <= rows
    u = HALF_STEP[got_o.dtype]
    tol = u * (o.abs() + A) * 1.01 + 2e-4 * A + 1e-30
    if got_o.dtype == torch.float16:
        tol = tol + 2.0 ** -25 * seen + 2.0 ** -25
    err = (got_o[:o.shape[0]].double() - o).abs()
    assert torch.isfinite(err).all(), f"{what}: non-finite outputs"
    over = (err / tol).max().item()
    assert over <= 1.0, f"{what}: error {over:.2f} times the bound"
    if got_lse2 is not None:
        e = (got_lse2[:o.shape[0]].double() - lse2).abs()
        # the score's error in exponent units (5.5e-5 * log2 e), 32-bit rounding of lse2 itself
        assert (e <= 1.5e-4 + 2.0 ** -23 * lse2.abs()).all(), f"{what}: lse2 off by {e.max().item():.2e}"
