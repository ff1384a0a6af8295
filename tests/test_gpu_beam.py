"""Beam search over a paged cache: the selection, the reordering of the beams' block tables, and both with plan, write and attention."""
import math
import random

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _clean():
    clis.clis_clear_device_error()
    yield
    torch.cuda.synchronize()
    assert clis.clis_get_device_error() == 0


# ------------------------------------------------------------------ selection


def reference(logits, scores, K):
    """(values in 64 bits, parent, token), best first, ties to the lowest place."""
    V = logits.shape[2]
    x = logits.double().cpu()
    v = (scores.double().cpu()[..., None] + (x - torch.logsumexp(x, -1, keepdim=True))).flatten(1)
    v = torch.where(v.abs() < math.inf, v, -math.inf)
    best, at = torch.sort(v, dim=-1, descending=True, stable=True)
    pad = max(0, K - best.shape[1])
    best = torch.nn.functional.pad(best, (0, pad), value=-math.inf)[:, :K]
    at = torch.nn.functional.pad(at, (0, pad))[:, :K]
    none = best == -math.inf
    return best, torch.where(none, -1, at // V).int(), torch.where(none, -1, at % V).int()


def check(logits, scores, K, got=None):
    """Places are equal; scores are off by the rounding to 32 bits and the sum's logarithm: its terms are off by 2^-22
    each, the 32-bit sums of up to 2^18 terms (in groups of 16 and 32) by 2^-19 at most: 4e-6 in all."""
    got = clis.beam_select(logits, scores, K) if got is None else got
    best, parent, token = reference(logits, scores, K)
    assert torch.equal(got.parent.cpu(), parent) and torch.equal(got.token.cpu(), token)
    live = best > -math.inf
    assert torch.equal(got.scores.cpu() > -math.inf, live)
    e = (got.scores.cpu().double() - best)[live].abs()
    assert (e <= 4e-6 + 2.0 ** -24 * best[live].abs()).all()
    return got


@pytest.mark.parametrize("R,W,V,K", [
    (1, 1, 1, 1), (1, 1, 1, 3), (2, 3, 2, 9), (3, 4, 511, 8), (2, 4, 512, 8), (2, 4, 513, 8), (1, 5, 1031, 10),
    (8, 4, 32003, 8), (2, 16, 50000, 32), (1, 64, 3000, 64), (3, 1, 131072, 64), (65, 8, 8192, 16), (1, 2, 300007, 4),
    (11, 15, 35, 14), (37, 7, 2397, 12), (8, 4, 50257, 64), (3, 14, 8, 17), (9, 40, 700, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_selection(R, W, V, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(R * 1000 + V)
    logits = (3 * torch.randn((R, W, V), generator=g, device="cuda")).to(DT[dtype])
    scores = -5 * torch.rand((R, W), generator=g, device="cuda")
    check(logits, scores, K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,levels", [(2000, 1), (5000, 3), (700, 2), (33000, 4)])
def test_ties(dtype, V, levels):
    """Few different logits, beams alike: thousands of equal values, within and across chunks and beams."""
    g = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randint(0, levels, (2, 4, V), generator=g, device="cuda").to(DT[dtype])
    logits[1] = logits[1, 0]
    scores = torch.zeros((2, 4), device="cuda")
    check(logits, scores, 64)
    check(logits, scores, 5)


def test_equal_rows_tie_whatever_their_alignment():
    g = torch.Generator(device="cuda").manual_seed(5)
    for dtype in DT.values():
        row = (4 * torch.randn(40009, generator=g, device="cuda")).to(dtype)
        logits = row.expand(1, 9, 40009).contiguous()  # rows at every alignment
        got = check(logits, torch.full((1, 9), -2.5, device="cuda"), 18)
        assert got.parent[0, :9].tolist() == list(range(9))


def test_masked_tokens_and_beams_not_in_use():
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = torch.randn((4, 3, 1000), generator=g, device="cuda").to(torch.bfloat16)
    scores = -torch.rand((4, 3), generator=g, device="cuda")
    logits[0, :, torch.rand(1000, generator=g, device="cuda") < 0.9] = -math.inf
    logits[1] = -math.inf
    logits[1, 2, 7] = 0.5          # one candidate in all
    scores[2] = -math.inf          # none
    scores[3, 1] = -math.inf
    got = check(logits, scores, 8)
    assert got.token[1].tolist() == [7] + [-1] * 7 and got.parent[2].tolist() == [-1] * 8


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,V", [(60, 20001), (60, 16384), (1100, 600)])
def test_runs_of_beams_in_use(R, V, dtype):
    """More logits than the GPU holds warps for: the beams in use are shared out among them, of up to 8,192 rows;
    a third is not in use, with NaN where nobody looks, among them the first and last rows and whole requests."""
    g = torch.Generator(device="cuda").manual_seed(R + V)
    logits = (3 * torch.randn((R, 8, V), generator=g, device="cuda")).to(DT[dtype])
    scores = -5 * torch.rand((R, 8), generator=g, device="cuda")
    dead = torch.rand((R, 8), generator=g, device="cuda") < 0.33
    dead[0, 0] = dead[-1, -1] = True
    dead[R // 2] = dead[R // 2 + 1] = True
    scores[dead] = -math.inf
    logits[dead] = math.nan
    check(logits, scores, 4)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_are_no_distribution(bad):
    g = torch.Generator(device="cuda").manual_seed(7)
    logits = torch.randn((1, 3, 5001), generator=g, device="cuda")
    scores = torch.zeros((1, 3), device="cuda")
    logits[0, 1, 4999] = bad
    got = check(logits, scores, 6)
    assert (got.parent != 1).all()
    scores[0, 0] = bad
    got = check(logits, scores, 6)
    assert (got.parent == 2).all()


def test_far_logits():
    """Logits in the thousands, sums of one term, and scores far below: the order is that of 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = 2000 * torch.randn((2, 4, 3000), generator=g, device="cuda")
    scores = -1000 * torch.rand((2, 4), generator=g, device="cuda")
    got = clis.beam_select(logits, scores, 16)
    best, parent, token = reference(logits, scores, 16)
    assert torch.equal(got.parent.cpu(), parent) and torch.equal(got.token.cpu(), token)
    # the output's own rounding, and that of the maximum's fp32 product with log2 e, which cancels
    assert ((got.scores.cpu().double() - best).abs() <= 4e-6 + 2.0 ** -24 * best.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [1000, 40009])
def test_masked_by_the_lowest_value(dtype, V):
    """Masks of the type's lowest number instead of -inf: such words are candidates behind all others, and a row of
    nothing else is as good as any constant one, log V below its score (in 64 bits the logarithm is lost beside such numbers,
    so the reference takes the maximum off first)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    low = torch.finfo(DT[dtype]).min
    logits = (3 * torch.randn((3, 4, V), generator=g, device="cuda")).to(DT[dtype])
    logits[:, :, torch.rand(V, generator=g, device="cuda") < 0.5] = low
    logits[1, 2] = low
    logits[2] = low
    scores = -torch.rand((3, 4), generator=g, device="cuda")
    scores[1, 2] = 12.0
    got = clis.beam_select(logits, scores, 40)
    x = logits.double().cpu()
    x = x - x.amax(-1, keepdim=True)
    v = (scores.double().cpu()[..., None] + (x - x.exp().sum(-1, keepdim=True).log())).flatten(1)
    best, at = torch.sort(v, dim=-1, descending=True, stable=True)
    best, at = best[:, :40], at[:, :40]
    assert torch.equal(got.parent.cpu(), (at // V).int()) and torch.equal(got.token.cpu(), (at % V).int())
    assert (got.parent[1] == 2).any() and got.token[2].tolist() == list(range(40))
    assert ((got.scores.cpu().double() - best).abs() <= 4e-6 + 2.0 ** -24 * best.abs()).all()


def test_strided_logits_and_no_requests():
    g = torch.Generator(device="cuda").manual_seed(9)
    big = torch.randn((3, 6, 2100), generator=g, device="cuda").to(torch.float16)
    check(big[:, ::2, 17:2017], -torch.rand((3, 3), generator=g, device="cuda"), 6)
    check(big[0].expand(2, 6, 2100), -torch.rand((2, 6), generator=g, device="cuda"), 6)
    got = clis.beam_select(torch.empty((0, 4, 100), device="cuda"), torch.empty((0, 4), device="cuda"))
    assert got.parent.shape == (0, 4)


def test_selection_in_a_graph():
    logits = torch.randn((4, 4, 5003), device="cuda").to(torch.bfloat16)
    scores = torch.zeros((4, 4), device="cuda")
    clis.beam_select(logits, scores, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = clis.beam_select(logits, scores, 8)
    for _ in range(3):
        logits.normal_()
        scores.uniform_(-3, 0)
        graph.replay()
        check(logits, scores, 8, got)


# ----------------------------------------------------------------- reordering


def beams(R, W, page, width, seed, free, dup=True):
    """Tables of requests whose beams share a random number of full pages (a tree: pairs of beams share more), lengths, and a ring."""
    rng = random.Random(seed)
    table = [[-1] * width for _ in range(R * W)]
    lens = [0] * (R * W)
    at = 0
    pages = list(range(R * W * width + free))
    rng.shuffle(pages)
    for r in range(R):
        n = rng.randint(0, width * page)
        shared = rng.randint(0, n // page) if dup else 0
        mid = rng.randint(shared, n // page) if dup else 0
        for w in range(W):
            if w and rng.random() < 0.15:
                continue  # a beam not in use
            m = n if rng.random() < 0.8 else rng.randint(mid * page, n)
            lens[r * W + w] = m
            for c in range(-(-m // page)):
                like = next((v for v in range(w) if c < -(-lens[r * W + v] // page) and lens[r * W + v]
                             and (c < shared or (c < mid and v // 2 == w // 2))), None)
                if like is not None:
                    table[r * W + w][c] = table[r * W + like][c]
                else:
                    table[r * W + w][c] = pages[at]
                    at += 1
    total = at + free
    used = sorted(pages[:at])
    ids = rng.sample(range(total), total)
    new = dict(zip(used, ids[:at]))
    table = [[new.get(p, -1) for p in row] for row in table]
    head = rng.randint(0, 5 * total)
    ring = [-1] * total
    for i, p in enumerate(ids[at:]):
        ring[(head + i) % total] = p
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"table": torch.tensor(table, **i32), "lens": torch.tensor(lens, **i32), "ring": torch.tensor(ring, **i32),
            "state": torch.tensor([head, head + free], dtype=torch.int64, device="cuda"), "pages": total}


def reorder_reference(b, parent, page, tensors):
    """The definition, in plain Python; copies the rows of `tensors` (CPU, [layers, pages, H, page, ...])."""
    table, lens, ring, (head, tail) = b["table"].tolist(), b["lens"].tolist(), b["ring"].tolist(), b["state"].tolist()
    R, W = len(parent), len(parent[0])
    width, F = len(table[0]), len(ring)
    avail, out, out_lens, done, gone, fits = tail - head, [], [], [], [], True
    h = head
    for r in range(R):
        rows = table[r * W:(r + 1) * W]
        have = [-(-lens[r * W + w] // page) for w in range(W)]
        again = [p >= 0 and p in parent[r][:w] and lens[r * W + p] % page != 0 for w, p in enumerate(parent[r])]
        fits = fits and h + sum(again) <= head + avail
        ok = fits or not any(again)
        done.append(int(ok))
        ps = parent[r] if ok else list(range(W))
        new = []
        for w, p in enumerate(ps):
            n = lens[r * W + p] if p >= 0 else 0
            row = (rows[p][:have[p]] if p >= 0 else [])
            if ok and again[w]:
                fresh = ring[h % F]
                h += 1
                for t in tensors:
                    t[:, fresh, :, :n % page] = t[:, row[-1], :, :n % page]
                row = row[:-1] + [fresh]
            out_lens.append(n)
            new.append(row + [-1] * (width - len(row)))
        out += new
        if ok:
            for c in range(width):
                named = {row[c] for row in new}
                seen = set()
                for w in range(W):
                    if c < have[w] and rows[w][c] not in named and rows[w][c] not in seen:
                        seen.add(rows[w][c])
                        gone.append(rows[w][c])
    for i, p in enumerate(gone):
        ring[(tail + i) % F] = p
    return out, out_lens, done, ring, [h, tail + len(gone)]


def run_reorder(b, parent, page, tensors, scales, in_place, W):
    cpu = [t.view(torch.int8).cpu() if t.element_size() == 1 else t.cpu() for t in tensors + scales]
    want = reorder_reference(b, parent.tolist(), page, cpu)
    r = clis.paged_reorder(b["lens"], parent, b["table"], b["ring"], b["state"], tensors, scales,
                           out=b["table"] if in_place else None, page_size=page)
    assert (r.block_table is b["table"]) == in_place
    assert r.block_table.tolist() == want[0] and r.lens.tolist() == want[1] and r.done.tolist() == want[2]
    assert b["ring"].tolist() == want[3] and r.ring_state.tolist() == want[4]
    for t, c in zip(tensors + scales, cpu):
        assert torch.equal((t.view(torch.int8) if t.element_size() == 1 else t).cpu(), c)
    return r


def parents(R, W, seed):
    rng = random.Random(seed)
    rows = []
    for r in range(R):
        kind = rng.randrange(4)
        rows.append([rng.randrange(W) for _ in range(W)] if kind else [rng.choice([-1, rng.randrange(W)]) for _ in range(W)])
        if rng.random() < 0.15:
            rows[-1] = [-1] * W
        if rng.random() < 0.15:
            rows[-1] = list(range(W))
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("R,W,page,width,kind", [
    (1, 1, 8, 3, "bf16"), (1, 4, 16, 5, "bf16"), (7, 3, 8, 9, "int8"), (20, 8, 16, 4, "e4m3"), (3, 64, 8, 12, "none"),
    (5, 5, 8, 700, "none"), (300, 2, 8, 2, "bf16"), (2, 33, 32, 3, "int8")])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder(R, W, page, width, kind, in_place):
    for seed in range(3):
        b = beams(R, W, page, width, seed + 10 * R, free=R * W + 2)
        L, H, d = 2, 3, 64
        shape = (L, b["pages"], H, page, d)
        tensors, scales = [], []
        if kind == "bf16":
            tensors = [torch.randn(shape, device="cuda").to(torch.bfloat16) for _ in range(2)]
        elif kind != "none":
            tensors = [torch.randint(-128, 127, shape, device="cuda", dtype=torch.int8) for _ in range(2)]
            tensors = [t.view(torch.float8_e4m3fn) for t in tensors] if kind == "e4m3" else tensors
            scales = [torch.rand(shape[:-1], device="cuda") for _ in range(2)]
        run_reorder(b, parents(R, W, seed), page, tensors, scales, in_place, W)


def test_too_few_pages():
    """Requests up to the first that the ring is too short for go on, those behind only without a copy; nothing is lost."""
    page = 8
    b = beams(12, 4, page, 6, 3, free=5, dup=True)
    b["lens"] = torch.where(b["lens"] > 3, b["lens"] - (b["lens"] % page == 0).int() * 3, b["lens"])  # partly filled
    par = torch.zeros((12, 4), dtype=torch.int32, device="cuda")
    par[5] = torch.arange(4)
    par[9] = -1
    r = run_reorder(b, par, page, [], [], False, 4)
    assert clis.clis_get_device_error() == clis.PAGED_POOL_BIT
    assert 0 < sum(r.done.tolist()) < 12
    clis.clis_clear_device_error()


def test_bad_inputs_leave_a_request_as_it_was():
    b = beams(4, 3, 8, 5, 1, free=20)
    par = torch.tensor([[0, 0, 0], [0, 3, 1], [1, 1, 1], [-7, 0, -1]], dtype=torch.int32, device="cuda")
    b["lens"][6] = 1 << 20
    r = clis.paged_reorder(b["lens"], par, b["table"], b["ring"], b["state"], page_size=8)
    assert r.done.tolist() == [1, 0, 0, 1]
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT | clis.PAGED_LENGTH_BIT
    assert torch.equal(r.lens[3:9], b["lens"][3:9])
    have = (b["lens"][3:6] + 7) // 8
    for w in range(3):
        assert torch.equal(r.block_table[3 + w, :have[w]], b["table"][3 + w, :have[w]])
    clis.clis_clear_device_error()
    # page numbers out of range: nothing is copied from or to them
    b = beams(1, 2, 8, 3, 2, free=4)
    b["lens"][:] = 20
    b["table"][0] = torch.tensor([0, 1, 1 << 30])
    k = torch.randn((1, b["pages"], 2, 8, 64), device="cuda").to(torch.bfloat16)
    before = k.clone()
    clis.paged_reorder(b["lens"], torch.zeros((1, 2), dtype=torch.int32, device="cuda"), b["table"], b["ring"], b["state"], [k])
    assert clis.clis_get_device_error() & clis.PAGED_INDEX_BIT and torch.equal(k, before)
    clis.clis_clear_device_error()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["negative length", "long", "parent", "pool"])
def test_a_refused_request_keeps_its_rows(what, in_place):
    """Whole rows, whatever is wrong with the request; its neighbours go on."""
    b = beams(3, 4, 8, 6, 5, free=0 if what == "pool" else 20)
    b["lens"][:] = torch.tensor([20, 20, 17, 9] * 3)
    b["table"][4:8, 3:] = torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3)  # (behind the pages: kept as well)
    par = torch.tensor([[0, 1, 2, 3], [0, 0, 3, 1], [3, 2, 1, 0]], dtype=torch.int32, device="cuda")
    if what == "parent":
        par[1, 2] = 4
    elif what != "pool":
        b["lens"][6] = -3 if what == "negative length" else 49
    table, lens = b["table"].clone(), b["lens"].clone()
    r = clis.paged_reorder(b["lens"], par, b["table"], b["ring"], b["state"], page_size=8, out=b["table"] if in_place else None)
    assert clis.clis_get_device_error() == {"parent": clis.PAGED_INDEX_BIT, "pool": clis.PAGED_POOL_BIT}.get(what, clis.PAGED_LENGTH_BIT)
    assert r.done.tolist() == [1, 0, 1]
    assert torch.equal(r.block_table[4:8], table[4:8]) and torch.equal(r.lens[4:8], lens[4:8])
    assert torch.equal(r.lens[8:], lens[8:].flip(0)) and torch.equal(r.block_table[8:, :2], table[8:, :2].flip(0))
    assert torch.equal(r.ring_state, b["state"])
    clis.clis_clear_device_error()


def test_strided_caches():
    """[pages, page_size, H, d] order, one layer of several, rows of 4-byte multiples only."""
    page, W = 8, 3
    b = beams(5, W, page, 4, 21, free=20)
    a = torch.randn((2, b["pages"], page, 3, 68), device="cuda").to(torch.bfloat16)
    k = a.transpose(2, 3)[..., 2:66]
    s = torch.rand((b["pages"], page, 3), device="cuda").transpose(1, 2)
    par = torch.tensor([[1, 1, 1], [0, 0, 2], [2, 2, 0], [0, 1, 2], [-1, 0, 0]], dtype=torch.int32, device="cuda")
    kc, sc = k.cpu().clone(), s.cpu().clone()[None]
    want = reorder_reference(b, par.tolist(), page, [kc, sc])
    r = clis.paged_reorder(b["lens"], par, b["table"], b["ring"], b["state"], [k], [s])
    assert r.block_table.tolist() == want[0] and torch.equal(k.cpu(), kc) and torch.equal(s.cpu()[None], sc)


# ------------------------------------------------------------ a search, whole


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8, torch.float8_e4m3fn])
def test_a_search(dtype):
    """Prompts of several requests, then a few steps of beam search with two layers over one cache, against beams that each
    keep a list of their own tokens' keys and values.  The cache's pages are all free again at the end."""
    g = torch.Generator(device="cuda").manual_seed(31)
    R, W, H, Hk, d, V, layers, page = 3, 4, 8, 2, 64, 203, 2, 8
    prompt = [13, 8, 21]
    cache = clis.PagedCache(layers=layers, num_pages=200, num_kv_heads=Hk, d=d, max_seqs=R * W, max_len=64, page_size=page, dtype=dtype)
    emb = torch.randn((V, (H + 2 * Hk) * d), generator=g, device="cuda").to(torch.bfloat16)
    head = 0.2 * torch.randn((H * d, V), generator=g, device="cuda")
    inv = 100.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    axis = torch.zeros(32, dtype=torch.int32, device="cuda")
    plain = torch.bfloat16

    def step(tokens, new, max_q):
        """Logits of the step's rows [T, V]."""
        T = tokens.numel()
        plan = cache.begin(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        out = 0
        for i in range(layers):
            x = emb[(tokens * (i + 3)) % V].reshape(T, H + 2 * Hk, d)
            q, k, v = (t.contiguous() for t in x.split([H, Hk, Hk], 1))
            out = out + cache.attend(i, q, k, v, plan, max_q, rope=(inv, axis)).float()
        return (out.reshape(T, -1) @ head)

    # the prompts, read by beam 0 of each request
    tokens = [torch.randint(0, V, (n,), generator=g, device="cuda") for n in prompt]
    new = [n if w == 0 else 0 for n in prompt for w in range(W)]
    lg = step(torch.cat(tokens), new, max(prompt))
    last = torch.tensor([sum(prompt[:r + 1]) - 1 for r in range(R)], device="cuda")
    scores = torch.full((R, W), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    logits = lg[last][:, None].expand(R, W, V)
    histories = [[t.tolist() for _ in range(W)] for t in tokens]

    def dense(hist):
        """Logits of one beam's last token from all of its tokens, in 64 bits; keys and values as a cache of `dtype` holds them."""
        t = torch.tensor(hist, device="cuda")
        n, out = len(hist), 0
        for i in range(layers):
            x = emb[(t * (i + 3)) % V].reshape(n, H + 2 * Hk, d)
            q, k, v = (y.contiguous() for y in x.split([H, Hk, Hk], 1))
            one = clis.PagedCache(layers=1, num_pages=9, num_kv_heads=Hk, d=d, max_seqs=1, max_len=64, page_size=page, dtype=dtype)
            p = one.begin(torch.tensor([n], dtype=torch.int32, device="cuda"), n)
            qr = clis.paged_append(k, v, one.k[0], one.v[0], p.slots, q=q, positions=p.positions, inv_freq=inv, axis=axis, **one._scales(0))
            if dtype == plain:
                k, v = one.read(0, p.cu_q, n)
                k, v = k.double(), v.double()
            else:
                at = p.slots
                k, v = ((c.view(torch.int8)[at // page, :, at % page].view(dtype).float() * s[at // page, :, at % page][..., None]).double()
                        for c, s in ((one.k[0], one.k_scale[0]), (one.v[0], one.v_scale[0])))
            k, v = (y.transpose(0, 1).repeat_interleave(H // Hk, 0) for y in (k, v))
            a = torch.softmax((qr[-1].double()[:, None] @ k.transpose(1, 2)) / math.sqrt(d), -1)
            out = out + (a @ v)[:, 0]
        return out.reshape(-1) @ head.double()

    for it in range(12):
        got = clis.beam_select(logits, scores, W)
        assert (got.token >= 0).all()
        assert cache.reorder(got.parent).tolist() == [1] * R
        scores = got.scores
        histories = [[histories[r][p] + [t] for p, t in zip(got.parent[r].tolist(), got.token[r].tolist())] for r in range(R)]
        assert cache.lens.tolist() == [len(h) - 1 for r in range(R) for h in histories[r]]
        lg = step(got.token.reshape(-1).long(), [1] * (R * W), 1)
        logits = lg.reshape(R, W, V)
        if it % 3 == 2:
            for r in range(R):
                for w in range(W):
                    want = dense(histories[r][w])
                    # two layers' outputs rounded to bf16 (2^-8 of each, weights too), 512 products with N(0, 0.2^2): the
                    # sum's error has a deviation of at most 0.2 * sqrt(512) * 2 * 2 * 2^-8 * 1.2; four of them
                    assert (logits[r, w].double() - want).abs().max().item() <= 4 * 0.2 * math.sqrt(512) * 4 * 2.0 ** -8 * 1.2
    assert cache.reorder(torch.full((R, W), -1, dtype=torch.int32, device="cuda")).tolist() == [1] * R
    head_, tail = cache.ring_state.tolist()
    assert tail - head_ == 200 and cache.lens.tolist() == [0] * (R * W)
    assert sorted(cache.ring[(head_ + torch.arange(200, device="cuda")) % 200].tolist()) == list(range(200))


def check_pages(cache):
    """Every page is free once or held by a row, and not both; rows share pages only in the same column."""
    page, (head, tail) = cache.page_size, cache.ring_state.tolist()
    F = cache.ring.numel()
    free = [cache.ring[i % F].item() for i in range(head, tail)]
    held = {(p, c) for n, row in zip(cache.lens.tolist(), cache.block_table.tolist()) for c, p in enumerate(row[:-(-n // page)])}
    assert sorted(free + [p for p, _ in held]) == list(range(F))


def test_beams_ended_by_the_plan():
    """Beams that share pages end by a negative length of the next step, some of them or all: a page is free once its last
    row has ended, and free once."""
    R, W = 2, 4
    cache = clis.PagedCache(layers=1, num_pages=50, num_kv_heads=1, d=64, max_seqs=R * W, max_len=64, page_size=8)

    def begin(*new):
        cache.begin(torch.tensor(new, dtype=torch.int32, device="cuda"), 40)
        check_pages(cache)

    def reorder(*parent):
        assert cache.reorder(torch.tensor(parent, dtype=torch.int32, device="cuda").view(R, W)).tolist() == [1] * R
        check_pages(cache)

    begin(21, 0, 0, 0, 16, 0, 0, 0)
    reorder(*[0] * 8)
    for _ in range(4):
        begin(*[1] * 8)
    reorder(0, 0, 2, 2, 1, 1, 1, 1)
    for _ in range(4):
        begin(*[1] * 8)
    begin(1, -1, 1, 1, -1, -1, 1, -1)                     # one of two that share, three of four, beside others that go on
    begin(-1, 0, -1, -1, 0, 0, 1, 0)                      # the rest of a request, one of them the last to name a page
    reorder(-1, -1, -1, -1, 2, 2, -1, 2)
    begin(5, 0, 0, 0, -2, -1, 0, 1)
    begin(-1, -1, -1, -1, -1, -1, -1, -1)
    assert cache.lens.tolist() == [0] * 8 and (cache.ring_state[1] - cache.ring_state[0]).item() == 50


@pytest.mark.parametrize("R,W,page,width", [(1, 2, 8, 3), (7, 4, 16, 9), (40, 8, 8, 30), (3, 64, 8, 6), (300, 3, 8, 5)])
def test_plan_of_beams_against_a_host_loop(R, W, page, width):
    """Pages given back, in the order of rows and columns: those that no row of the request names any more that goes on
    or is finished before; rows that go on take theirs as ever."""
    for seed in range(3):
        rng = random.Random(seed)
        b = beams(R, W, page, width, seed + 100 * R, free=R * W + 1)
        cap, lens, table = width * page, b["lens"].tolist(), b["table"].tolist()
        new = [rng.choice([-1, -1, 0, min(rng.randint(0, page), cap - n)]) for n in lens]
        if seed == 2:
            new = [-1] * (R * W)
        have, (head, tail), F = [-(-n // page) for n in lens], b["state"].tolist(), b["pages"]
        ring, h = b["ring"].tolist(), head
        for s, n in enumerate(new):
            for c in range(have[s], -(-(lens[s] + n) // page) if n > 0 else 0):
                table[s][c] = ring[h % F]
                h += 1
        for s, n in enumerate(new):
            r0 = s - s % W
            for c in range(have[s] if n < 0 else 0):
                if not any(v != s and (new[v] >= 0 or v < s) and c < have[v] and table[v][c] == table[s][c] for v in range(r0, r0 + W)):
                    ring[tail % F] = table[s][c]
                    tail += 1
        p = clis.paged_plan(b["lens"], torch.tensor(new, dtype=torch.int32, device="cuda"), b["table"], b["ring"], b["state"], page,
                            sum(max(n, 0) for n in new), beams=W)
        assert p.ring_state.tolist() == [h, tail] and b["ring"].tolist() == ring and b["table"].tolist() == table
        assert p.kv_len.tolist() == [n + m if m >= 0 else 0 for n, m in zip(lens, new)]


def test_requests_of_another_number_of_beams():
    """A cache that served requests of three beams serves requests of two: rows 2 and 3 share pages then."""
    cache = clis.PagedCache(layers=1, num_pages=40, num_kv_heads=1, d=64, max_seqs=6, max_len=64, page_size=8)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    for W in (3, 2):
        cache.begin(torch.tensor([17 if r % W == 0 else 0 for r in range(6)], **i32), 60)
        assert cache.reorder(torch.zeros((6 // W, W), **i32)).tolist() == [1] * (6 // W)
        cache.begin(torch.ones(6, **i32), 6)
        check_pages(cache)
        cache.begin(torch.tensor([-1, 1, -1, 0, 1, -1], **i32), 6)
        check_pages(cache)
        cache.begin(torch.full((6,), -1, **i32), 6)
        check_pages(cache)


def test_a_step_of_the_search_in_a_graph():
    """Plan, write, attention, selection and reordering captured once and replayed, against the same steps made one by one."""
    R, W, H, Hk, d, V = 2, 3, 4, 2, 64, 1000
    g = torch.Generator(device="cuda").manual_seed(41)
    emb = torch.randn((V, (H + 2 * Hk) * d), generator=g, device="cuda").to(torch.bfloat16)
    head = 0.2 * torch.randn((H * d, V), generator=g, device="cuda")

    def fresh():
        cache = clis.PagedCache(layers=1, num_pages=60, num_kv_heads=Hk, d=d, max_seqs=R * W, max_len=64, page_size=8, dtype=torch.int8)
        x = emb[:20].reshape(20, H + 2 * Hk, d)
        plan = cache.begin(torch.tensor([9, 0, 0, 11, 0, 0], dtype=torch.int32, device="cuda"), 20)
        cache.attend(0, *(t.contiguous() for t in x.split([H, Hk, Hk], 1)), plan, 11)
        cache.reorder(torch.zeros((R, W), dtype=torch.int32, device="cuda"))
        return cache, torch.arange(R * W, device="cuda"), torch.zeros((R, W), device="cuda")

    one = torch.ones(R * W, dtype=torch.int32, device="cuda")

    def step(cache, token, scores):
        x = emb[token].reshape(R * W, H + 2 * Hk, d)
        plan = cache.begin(one, R * W)
        o = cache.attend(0, *(t.contiguous() for t in x.split([H, Hk, Hk], 1)), plan, 1)
        got = clis.beam_select((o.reshape(R * W, -1).float() @ head).reshape(R, W, V), scores, W)
        cache.reorder(got.parent)
        token.copy_(got.token.reshape(-1))
        scores.copy_(got.scores)

    a, b = fresh(), fresh()
    warm = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*b)
    for _ in range(8):
        step(*a)
        graph.replay()
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2]) and torch.equal(a[0].lens, b[0].lens)
        assert torch.equal(a[0].block_table, b[0].block_table) and torch.equal(a[0].ring_state, b[0].ring_state)


def test_logits_beyond_32_bits():
    """2.2 * 10^9 logits in all: the last request's place is past 2^32 bytes and 2^31 values."""
    R, W, V = 70, 8, 4000037
    logits = torch.empty((R, W, V), dtype=torch.bfloat16, device="cuda").fill_(-3.0)
    g = torch.Generator(device="cuda").manual_seed(42)
    scores = -torch.rand((R, W), generator=g, device="cuda")
    logits[::23] = torch.randn((W, V), generator=g, device="cuda").to(torch.bfloat16)
    logits[R - 1] = torch.randn((W, V), generator=g, device="cuda").to(torch.bfloat16)
    got = clis.beam_select(logits, scores, 9)
    for r in (0, 1, 46, R - 1):
        check(logits[r:r + 1], scores[r:r + 1], 9, clis.BeamChoice(*(t[r:r + 1] for t in got)))


def test_refusals_on_the_host():
    x, s = torch.zeros((2, 3, 50), device="cuda"), torch.zeros((2, 3), device="cuda")
    for logits, scores, num, match in ((x[..., ::2], s, 3, "contiguous last"), (x.double(), s, 3, "bfloat16, float16 or float32"),
                                       (x, s[:1], 3, "scores"), (x, s.double(), 3, "scores"), (x, s, 0, "positive"), (x, s, 65, "UNSUPPORTED"),
                                       (x[:, :0], s[:, :0], 3, "beams and tokens")):
        with pytest.raises((ValueError, clis.ClisError), match=match):
            clis.beam_select(logits, scores, num)
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    st = torch.tensor([0, 10], dtype=torch.int64, device="cuda")
    k = torch.zeros((10, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    for args, kw, match in (((i(6), i(2, 3), i(6, 4), i(10), st, [k[0]]), {}, "4 or 5"), ((i(5), i(2, 3), i(6, 4), i(10), st, [k]), {}, "lens"),
                            ((i(6), i(2, 3), i(5, 4), i(10), st, [k]), {}, "block_table"), ((i(6), i(2, 3), i(6, 4), i(10), st, [k, k[:5]]), {}, "one size"),
                            ((i(6), i(2, 3), i(6, 4), i(10), st.int(), [k]), {}, "ring_state"), ((i(6), i(2, 3), i(6, 4), i(10), st, [k]), {"out": i(6, 5)}, "out"),
                            ((i(6), i(2, 3), i(6, 4), i(10), st, [k], [k[..., 0]]), {}, "MISALIGNED|multiple|aligned|INVALID")):
        with pytest.raises((ValueError, clis.ClisError), match=match):
            clis.paged_reorder(*args, **kw)
    with pytest.raises(TypeError):
        clis.paged_reorder(i(6), i(2, 3), i(6, 4), i(10), st, [1])
