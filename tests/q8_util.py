"""Inputs and 64-bit references for the tests of a cache held in 8 bits (no method code)."""
import math
import random

import torch

from paged_util import HALF_STEP

CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


def raw(t):
    """The codes' bytes (indexing a float8 tensor needs them)."""
    return t.view(torch.int8)


def make_q8(ctx, new, H, Hkv, d, page, dtype, code, seed=0, device="cuda", extra_rows=0, layout="hnd", spread=0.4, poison=True,
            columns=0):
    """Random batch over a paged cache of codes.  Pages are scattered; with ``poison`` the scales (and E4M3 codes)
    of rows that hold no key are NaN, int8 codes 111, and unused block-table entries out of range.  ``spread``: of
    the scales' logarithm.  ``columns``: further ones of the block table (by what it can hold a batch's kernels are chosen)."""
    g = torch.Generator(device=device).manual_seed(seed)
    rng = random.Random(seed)
    S, kv = len(ctx), [c + n for c, n in zip(ctx, new)]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    ids = list(range(pages))
    rng.shuffle(ids)
    bt = torch.full((S, max(need + [0]) + 2 + columns), 0x3FFFFFFF if poison else -1, dtype=torch.int32)
    shape = (pages, Hkv, page, d) if layout == "hnd" else (pages, page, Hkv, d)
    fill = 127 if code == "e4m3" else 111
    kc, vc = (torch.full(shape, fill if poison else 0, dtype=torch.int8, device=device) for _ in range(2))
    ks, vs = (torch.full(shape[:3], float("nan") if poison else 0.0, device=device) for _ in range(2))
    if layout != "hnd":
        kc, vc, ks, vs = (t.transpose(1, 2) for t in (kc, vc, ks, vs))
    keys, at = [], 0
    for s in range(S):
        mine, both = ids[at:at + need[s]], []
        at += need[s]
        bt[s, :need[s]] = torch.tensor(mine, dtype=torch.int32)
        for cache, scale in ((kc, ks), (vc, vs)):
            c = (torch.randn((kv[s], Hkv, d), generator=g, device=device) * (TOP[code] / 3)).clamp(-TOP[code], TOP[code]).round()
            c = raw(c.to(CODES[code]))
            x = torch.exp(spread * torch.randn((kv[s], Hkv), generator=g, device=device)) * (3 / TOP[code])
            for i, p in enumerate(mine):
                n = min(page, kv[s] - i * page)
                cache[p, :, :n] = c[i * page:i * page + n].transpose(0, 1)
                scale[p, :, :n] = x[i * page:i * page + n].transpose(0, 1)
            both.append((c.view(CODES[code]), x))
        keys.append(both)
    T = sum(new) + extra_rows
    q = torch.randn((T, H, d), generator=g, device=device).to(dtype)
    return {"q": q, "k_cache": kc.view(CODES[code]), "v_cache": vc.view(CODES[code]), "k_scale": ks, "v_scale": vs,
            "block_table": bt.to(device), "cu_q": torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device=device),
            "kv_len": torch.tensor(kv, dtype=torch.int32, device=device), "keys": keys, "ctx": ctx, "new": new,
            "max_q": max(new + [1]), "code": code}


def few_rows(b):
    """Query rows up to which a sequence of the batch runs the kernel for few rows (include/clis.h)."""
    S, width = b["block_table"].shape
    pages, Hkv, page, d = b["k_cache"].shape
    g, max_q = b["q"].shape[1] // Hkv, min(b["max_q"], b["q"].shape[0])
    rows, tile, keys = max_q * g, 24 if d == 64 else 16, 4096 // d
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if rows <= 64:
        return rows
    units = -(-width * page // keys) * S * Hkv * -(-rows // tile)
    if max_q <= 2048 and rows <= 2048 and units <= (6 if d == 64 else 17) * sms * 8:
        return rows
    if S * Hkv <= 4 * sms and 2 * S * Hkv * width * page * d <= 16 << 20:
        return 0
    return g if g <= 64 else 0


def check_q8(got_o, got_lse2, b, causal=True, scale=None, what=""):
    """Element-wise bounds derived from the arithmetic, per sequence.

    Few rows (values are code * scale exactly): the output is rounded once (u |o|); a weight times V's scale is
    rounded to fp16 once (2^-11 of A := sum p |v| / sum p) or, below 2^-14 of its shift, by up to 2^-25 where the largest
    stands at 2^7 (2^-32 max(p vs) sum |vc| / sum p); a score is a 32-bit dot product of d exact products, off by at
    most d 2^-24 sum |q k| scale, at 3 sigma of the scales' spread 4 times the unit normals' 5.5e-5, and is then multiplied by
    two factors (2^-23 of x, below 50): 3e-4 in the exponent, twice that times A; lg2, ex2 and the sums some 1e-6.
    Chunks: V's values are rounded to the data type first, which the reference does too; the rest as in paged_util, with
    the scores' error above."""
    q = b["q"]
    H, d = q.shape[1:]
    Hkv = b["k_cache"].shape[1]
    g = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = HALF_STEP[q.dtype]
    r0 = 0
    for s, (c, n) in enumerate(zip(b["ctx"], b["new"])):
        if n == 0:
            continue
        few = n * g <= few_rows(b)
        (kc, ks), (vc, vs) = b["keys"][s]
        k, v = kc.float().double() * ks.double()[..., None], vc.float().double() * vs.double()[..., None]
        if not few:
            v = (vc.float() * vs[..., None]).to(q.dtype).double()
        rep = lambda t: t.transpose(0, 1).repeat_interleave(g, 0)  # noqa: E731
        k, v, vcd, vsd = rep(k), rep(v), rep(vc.float().double().abs()), rep(vs.double())
        x = q[r0:r0 + n].double().transpose(0, 1) @ k.transpose(1, 2) * scale
        if causal:
            hide = torch.arange(c + n, device=q.device)[None] > torch.arange(c, c + n, device=q.device)[:, None]
            x = x.masked_fill(hide, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        L = p.sum(-1, keepdim=True)
        o, A = p @ v / L, p @ v.abs() / L
        if few:
            mw = (p * vsd[:, None]).amax(-1, keepdim=True)
            tol = u * o.abs() + (2.0 ** -11 + 6e-4) * A * 1.01 + 2.0 ** -32 * mw * ((p > 0).double() @ vcd) / L
        else:
            tol = u * (o.abs() + A) * 1.01 + 8e-4 * A
            if q.dtype == torch.float16:
                tol = tol + 2.0 ** -25 * ((p > 0).double() @ v.abs())
        if q.dtype == torch.float16:
            tol = tol + 2.0 ** -25
        e = (got_o[r0:r0 + n].double().transpose(0, 1) - o).abs()
        assert torch.isfinite(e).all(), f"{what}: sequence {s}: non-finite outputs"
        over = (e / (tol + 1e-30)).max().item()
        assert over <= 1.0, f"{what}: sequence {s} ({'few rows' if few else 'chunk'}): error {over:.2f} times the bound"
        if got_lse2 is not None:
            ref = (m + L.log())[..., 0] / math.log(2.0)
            e = (got_lse2[r0:r0 + n].double().transpose(0, 1) - ref).abs()
            assert (e <= 6e-4 + 2.0 ** -22 * ref.abs()).all(), f"{what}: sequence {s}: lse2 off by {e.max().item():.2e}"
        r0 += n
