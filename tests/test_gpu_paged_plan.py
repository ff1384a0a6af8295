"""The plan of a serving step against a plain host computation, and whole steps through PagedCache."""
import random

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis
from paged_util import check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    clis.clis_clear_device_error()
    yield
    assert clis.clis_get_device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def host_plan(ctx, new, table, ring, head, tail, page, T):
    """The same step in plain Python; changes table and ring."""
    cu, kv, slots, pos, F = [0], [], [], [], len(ring)
    back = tail
    for s, (c, n) in enumerate(zip(ctx, new)):
        have = -(-c // page)
        if n < 0:
            for i in range(have):
                ring[back % F] = table[s][i]
                back += 1
            n, kvs = 0, 0
        else:
            for i in range(have, -(-(c + n) // page)):
                table[s][i] = ring[head % F]
                head += 1
            kvs = c + n
        for j in range(c, c + n):
            slots.append(table[s][j // page] * page + j % page)
            pos.append(j)
        cu.append(cu[-1] + n)
        kv.append(kvs)
    slots += [-1] * (T - len(slots))
    pos += [0] * (T - len(pos))
    return cu, kv, slots, pos, [head, back]


@pytest.mark.parametrize("S,page,big,seed", [(1, 8, 30, 0), (1, 16, 5000, 1), (5, 64, 300, 2), (33, 8, 100, 3), (700, 16, 90, 4),
                                            (1024, 32, 700, 5), (3000, 16, 40, 6), (16384, 8, 20, 7)])
def test_against_a_host_loop(S, page, big, seed):
    rng = random.Random(seed)
    ctx = [rng.choice([0, page, rng.randint(0, big), rng.randint(0, 10 * page)]) for _ in range(S)]
    new = [rng.choice([-1, 0, 1, 1, page, rng.randint(0, big)]) for _ in range(S)]
    have = [-(-c // page) for c in ctx]
    need = [max(h, -(-(c + max(n, 0)) // page)) for h, c, n in zip(have, ctx, new)]
    pages, width = sum(need) + 7, max(need) + 2
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[-1] * width for _ in range(S)]
    at = 0
    for s in range(S):
        table[s][:have[s]] = ids[at:at + have[s]]
        at += have[s]
    head = rng.randint(0, 10 ** 12)
    ring = [-1] * pages
    free = ids[at:]
    for i, p in enumerate(free):
        ring[(head + i) % pages] = p
    T = sum(max(n, 0) for n in new) + rng.choice([0, 0, 13])
    wide = torch.full((S, width + 3), -9, dtype=torch.int32, device="cuda")
    bt = wide[:, :width]
    bt.copy_(i32(table))
    dring = i32(ring)
    state = torch.tensor([head, head + len(free)], dtype=torch.int64, device="cuda")
    p = clis.paged_plan(i32(ctx), i32(new), bt, dring, state, page, T)
    cu, kv, slots, pos, after = host_plan(ctx, new, table, ring, head, head + len(free), page, T)
    assert p.cu_q.tolist() == cu and p.kv_len.tolist() == kv
    assert p.slots.tolist() == slots and p.positions.tolist() == pos
    assert p.ring_state.tolist() == after and state.tolist() == [head, head + len(free)]
    assert bt.tolist() == table and dring.tolist() == ring
    assert (wide[:, width:] == -9).all()


def test_no_sequences_and_no_tokens():
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    state = torch.tensor([0, 4], dtype=torch.int64, device="cuda")
    p = clis.paged_plan(none, none, none.reshape(0, 3), i32([0, 1, 2, 3]), state, 16, 5)
    assert p.cu_q.tolist() == [0] and p.slots.tolist() == [-1] * 5 and p.ring_state.tolist() == [0, 4]
    p = clis.paged_plan(i32([3]), i32([0]), i32([[2, -1]]), i32([0, 1, 2, 3]), state, 16, 0)
    assert p.cu_q.tolist() == [0, 0] and p.kv_len.tolist() == [3] and p.slots.numel() == 0


def test_out_of_pages_and_lengths():
    """A ring that runs out gives slots of -1 to what has no page, and is recorded; nothing else is touched."""
    state = torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    bt = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    p = clis.paged_plan(i32([0, 0]), i32([8, 9]), bt, i32([5, 6, 7, 8, 9, 10, 11, 12]), state, 8, 17, num_pages=100)
    assert clis.clis_get_device_error() == clis.PAGED_POOL_BIT
    clis.clis_clear_device_error()
    assert p.slots.tolist() == [40 + i for i in range(8)] + [-1] * 9 and p.ring_state.tolist() == [1, 1]
    assert bt.tolist() == [[5, -1, -1, -1], [-1, -1, -1, -1]]
    # lengths beyond the block table, more tokens than rows, a page number out of range
    for ctx, new, T, bit in ((40, 1, 1, clis.PAGED_LENGTH_BIT), (0, 33, 33, clis.PAGED_LENGTH_BIT), (-1, 1, 1, clis.PAGED_LENGTH_BIT),
                             (0, 9, 5, clis.PAGED_LENGTH_BIT), (2, 1, 1, clis.PAGED_INDEX_BIT)):
        bt = torch.full((1, 4), 99, dtype=torch.int32, device="cuda")
        state = torch.tensor([0, 8], dtype=torch.int64, device="cuda")
        p = clis.paged_plan(i32([ctx]), i32([new]), bt, i32([0, 1, 2, 3, 4, 5, 6, 7]), state, 8, T)
        assert clis.clis_get_device_error() & bit
        clis.clis_clear_device_error()
        assert max(p.slots.tolist()) < 64 and p.cu_q[1].item() <= T
    # counters that contradict the ring's size
    state = torch.tensor([5, 2], dtype=torch.int64, device="cuda")
    p = clis.paged_plan(i32([0]), i32([1]), bt, i32([0, 1, 2]), state, 8, 1)
    assert clis.clis_get_device_error() & clis.PAGED_POOL_BIT and p.slots.tolist() == [-1]
    clis.clis_clear_device_error()


@pytest.mark.parametrize("dtype,d,page,rotate", [(torch.bfloat16, 128, 16, True), (torch.float16, 64, 64, False)])
def test_steps_together(dtype, d, page, rotate):
    """Prompts, decoding, drafted tokens, a finished sequence whose pages are used again, over two
    layers: plan, write and attention as they are used, against softmax over all tokens so far."""
    H, Hk, S, layers = 8, 2, 4, 2
    cache = clis.PagedCache(layers, num_pages=60, num_kv_heads=Hk, d=d, max_seqs=S, max_len=40 * page, page_size=page, dtype=dtype)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    axis = torch.zeros(d // 2, dtype=torch.int32, device="cuda")
    hist = [[[torch.zeros(0, Hk, d, dtype=dtype, device="cuda")] * 2 for _ in range(S)] for _ in range(layers)]
    lens = [0] * S
    g = torch.Generator(device="cuda").manual_seed(d)
    for new, pad in (([50, 0, 170, 3], 0), ([1, 20, 1, 1], 5), ([1, 1, 1, 1], 0), ([4, 1, -1, 0], 2), ([1, 1, 90, 2], 0), ([1, 1, 1, 1], 3)):
        T = sum(max(n, 0) for n in new) + pad
        plan = cache.begin(i32(new), T)
        ctx = [0 if n < 0 else c for c, n in zip(lens, new)]
        n0 = [max(n, 0) for n in new]
        for layer in range(layers):
            q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(dtype) for h in (H, Hk, Hk))
            o = cache.attend(layer, q, k, v, plan, max(n0), rope=(inv, axis) if rotate else None)
            if rotate:
                q, k = (t[0].transpose(0, 1) for t in clis.rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None],
                                                                 plan.positions[:, None], inv, axis))
            at = 0
            for s, n in enumerate(new):
                if n < 0:
                    hist[layer][s] = [t[:0] for t in hist[layer][s]]
                    continue
                hist[layer][s] = [torch.cat((t, x[at:at + n])) for t, x in zip(hist[layer][s], (k, v))]
                at += n
            b = {"q": q, "k_cache": cache.k[layer], "ctx": ctx, "new": n0, "keys": [h[0] for h in hist[layer]],
                 "vals": [h[1] for h in hist[layer]]}
            check_attention(o, None, b)
        lens = [0 if n < 0 else c + n for c, n in zip(lens, new)]
        assert cache.lens.tolist() == lens
    used = sum(-(-n // page) for n in lens)
    head, tail = cache.ring_state.tolist()
    assert tail - head == 60 - used


def test_step_captured_and_replayed():
    """One captured step (plan, rotation and write, attention) serves steps of other lengths."""
    H, Hk, d, page, S, T = 4, 2, 64, 8, 3, 6
    inv = (10000.0 ** (-torch.arange(8, dtype=torch.float64) / 8)).cuda()
    axis = torch.zeros(8, dtype=torch.int32, device="cuda")

    def fresh():
        return clis.PagedCache(1, num_pages=30, num_kv_heads=Hk, d=d, max_seqs=S, max_len=80, page_size=page)

    def step(cache, new, q, k, v, out):
        plan = cache.begin(new, T)
        return cache.attend(0, q, k, v, plan, T, rope=(inv, axis), out=out)

    g = torch.Generator(device="cuda").manual_seed(9)
    steps = [(lens, [torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hk, Hk)])
             for lens in ([2, 3, 1], [1, 1, 1], [1, -1, 4], [1, 5, 0])]
    eager = fresh()
    want = [step(eager, i32(n), *x, torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")) for n, x in steps]
    cache, new, out = fresh(), i32([0, 0, 0]), torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    bufs = [torch.zeros_like(t) for t in steps[0][1]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, new, *bufs, out)
    for (n, x), w in zip(steps, want):
        new.copy_(i32(n))
        for b, t in zip(bufs, x):
            b.copy_(t)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert torch.equal(cache.lens, eager.lens) and torch.equal(cache.block_table, eager.block_table)


@pytest.mark.parametrize("S,page,seed", [(1, 8, 0), (6, 16, 1), (40, 8, 2), (900, 8, 3), (2000, 16, 4)])
@pytest.mark.parametrize("short", ["pages", "rows", "both"])
def test_what_cannot_be_served_stays_as_it_was(S, page, seed, short):
    """Too few free pages, or rows: the sequences from the first that lacks any on take no page, and those of
    them that need one (or rows that are not there) keep their length; nothing of them is written."""
    rng = random.Random(seed)
    ctx = [rng.randint(0, 6 * page) for _ in range(S)]
    new = [rng.choice([0, 1, 2, page, 3 * page, -1]) if S > 1 else 2 * page + 1 for _ in range(S)]
    have = [-(-c // page) for c in ctx]
    take = [max(0, -(-(c + max(n, 0)) // page) - h) for h, c, n in zip(have, ctx, new)]
    free = sum(take) * 2 // 3 if short != "rows" else sum(take) + 3
    T = sum(max(n, 0) for n in new)
    T = T * 3 // 5 if short != "pages" else T + 2
    pages, width = sum(have) + free, 12
    table, at = [[-1] * width for _ in range(S)], 0
    for s in range(S):
        table[s][:have[s]] = range(at, at + have[s])
        at += have[s]
    head = 5
    size = pages + 1
    ring = [-1] * size
    for i in range(free):
        ring[(head + i) % size] = at + i
    bt, dring = i32(table), i32(ring)
    p = clis.paged_plan(i32(ctx), i32(new), bt, dring, torch.tensor([head, head + free], dtype=torch.int64, device="cuda"),
                        page, T, num_pages=pages)
    cu, kv, slots, used, tail, first = [0], [], [-1] * T, 0, head + free, None
    for s in range(S):
        n = max(new[s], 0)
        rows, room = cu[-1] + n <= T, used + take[s] <= free
        if first is None and n > 0 and not (rows and room):
            first = s
        ok = n == 0 or (rows and (first is None or take[s] == 0))
        if new[s] < 0:
            for i in range(have[s]):
                ring[tail % size] = table[s][i]
                tail += 1
        elif ok:
            for i in range(take[s]):
                table[s][have[s] + i] = ring[(head + used + i) % size]
            used += take[s]
            for j in range(n):
                slots[cu[-1] + j] = table[s][(ctx[s] + j) // page] * page + (ctx[s] + j) % page
        kv.append(0 if new[s] < 0 else ctx[s] + n if ok else ctx[s])
        cu.append(cu[-1] + n)
    assert first is not None
    bit = (clis.PAGED_POOL_BIT if short != "rows" else 0) | (clis.PAGED_LENGTH_BIT if short != "pages" else 0)
    assert clis.clis_get_device_error() == bit
    clis.clis_clear_device_error()
    assert p.cu_q.tolist() == [min(c, T) for c in cu] and p.kv_len.tolist() == kv and p.slots.tolist() == slots
    assert p.ring_state.tolist() == [head + used, tail] and bt.tolist() == table and dring.tolist() == ring


def test_a_full_cache_goes_on():
    """Tokens that no page was left for are brought again once another sequence has finished; no page is lost."""
    cache = clis.PagedCache(1, num_pages=6, num_kv_heads=1, d=64, max_seqs=3, max_len=64, page_size=8)
    cache.begin(i32([16, 16, 8]), 40)
    plan = cache.begin(i32([1, 9, 1]), 11)          # one page is left: for the first sequence
    assert clis.clis_get_device_error() == clis.PAGED_POOL_BIT
    clis.clis_clear_device_error()
    assert cache.lens.tolist() == [17, 16, 8] and plan.slots.tolist()[1:] == [-1] * 10
    plan = cache.begin(i32([-1, 0, 0]), 0)
    plan = cache.begin(i32([0, 9, 1]), 10)
    assert cache.lens.tolist() == [0, 25, 9] and min(plan.slots.tolist()) >= 0
    cache.begin(i32([0, -1, -1]), 0)
    head, tail = cache.ring_state.tolist()
    assert tail - head == 6 and sorted(cache.ring.tolist()) == list(range(6))


def test_what_is_no_page_is_recorded():
    """In the ring, or given back."""
    state = torch.tensor([0, 2], dtype=torch.int64, device="cuda")
    for page in (-1, 4):
        p = clis.paged_plan(i32([0]), i32([9]), i32([[-1, -1]]), i32([3, page, 0, 0]), state, 8, 9)
        assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT and p.slots.tolist() == [24 + i for i in range(8)] + [-1]
        clis.clis_clear_device_error()
        clis.paged_plan(i32([9]), i32([-1]), i32([[1, page]]), i32([3, 2, 0, 0]), state, 8, 0)
        assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
        clis.clis_clear_device_error()


@pytest.mark.parametrize("S,page,seed", [(3, 8, 0), (7, 16, 1), (60, 8, 2), (1100, 16, 3)])
def test_a_full_table_row_concerns_nobody_else(S, page, seed):
    """Sequences that their block-table row cannot hold (or whose cached length is out of range), among others:
    they take no page, get no slot and keep their length; the others' rows stay where they were packed."""
    rng = random.Random(seed)
    width = 4
    cap = width * page
    ctx = [rng.choice([cap, cap, cap - 1, rng.randint(0, cap), rng.randint(0, page), 0]) for _ in range(S)]
    new = [rng.choice([1, 1, 2, cap + 1 - c if c else cap + 1, page, 0, -1]) for c in ctx]
    ctx[1], new[1] = cap, 1
    if S > 50:
        ctx[40], ctx[41], new[40], new[41] = -3, cap + 5, 2, 1   # lengths that cannot be
    held = [min(max(c, 0), cap) for c in ctx]
    full = [c != h or max(n, 0) > cap - h for c, h, n in zip(ctx, held, new)]
    have = [-(-c // page) for c in held]
    take = [0 if f else -(-(c + max(n, 0)) // page) - h for f, c, n, h in zip(full, held, new, have)]
    pages = sum(have) + sum(take) + 2
    table, at = [[-1] * width for _ in range(S)], 0
    for s in range(S):
        table[s][:have[s]] = range(at, at + have[s])
        at += have[s]
    free = pages - at
    ring = list(range(at, pages)) + [-1] * at
    T = sum(max(n, 0) for n in new) + 3
    bt, dring = i32(table), i32(ring)
    p = clis.paged_plan(i32(ctx), i32(new), bt, dring, torch.tensor([0, free], dtype=torch.int64, device="cuda"), page, T)
    assert clis.clis_get_device_error() == clis.PAGED_LENGTH_BIT
    clis.clis_clear_device_error()
    cu, kv, slots, head, tail = [0], [], [-1] * T, 0, free
    for s in range(S):
        n = max(new[s], 0)
        if new[s] < 0:
            for i in range(have[s]):
                ring[tail % pages] = table[s][i]
                tail += 1
        elif not full[s]:
            for i in range(take[s]):
                table[s][have[s] + i] = ring[head]
                head += 1
            for j in range(n):
                slots[cu[-1] + j] = table[s][(ctx[s] + j) // page] * page + (ctx[s] + j) % page
        kv.append(0 if new[s] < 0 else held[s] if full[s] else ctx[s] + n)
        cu.append(cu[-1] + n)
    assert p.cu_q.tolist() == cu and p.kv_len.tolist() == kv and p.slots.tolist() == slots
    assert p.ring_state.tolist() == [head, tail] and bt.tolist() == table and dring.tolist() == ring
    pos = p.positions.tolist()
    for s in range(S):
        if not full[s]:
            assert pos[cu[s]:cu[s + 1]] == list(range(ctx[s], ctx[s] + max(new[s], 0)))


def test_a_sequence_at_its_end_leaves_the_others_alone():
    """One of three sequences reaches max_len: the others' keys, values and outputs are those of a cache without it."""
    H, Hk, d, page = 4, 2, 64, 8
    g = torch.Generator(device="cuda").manual_seed(21)
    cache = clis.PagedCache(1, num_pages=30, num_kv_heads=Hk, d=d, max_seqs=3, max_len=16, page_size=page)
    hist = [[torch.zeros(0, Hk, d, dtype=torch.bfloat16, device="cuda")] * 2 for _ in range(3)]
    lens = [0, 0, 0]
    for new in ([5, 15, 9], [1, 1, 1], [2, 1, 1], [1, 3, 2]):
        T = sum(new)
        q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hk, Hk))
        plan = cache.begin(i32(new), T)
        o = cache.attend(0, q, k, v, plan, max(new))
        stays = [c + n > 16 for c, n in zip(lens, new)]
        assert clis.clis_get_device_error() == (clis.PAGED_LENGTH_BIT if any(stays) else 0)
        clis.clis_clear_device_error()
        at, rows, seqs = 0, [], []
        ctx = list(lens)
        for s, n in enumerate(new):
            if not stays[s]:
                hist[s] = [torch.cat((t, x[at:at + n])) for t, x in zip(hist[s], (k, v))]
                rows += range(at, at + n)
                seqs.append(s)
                lens[s] += n
            at += n
        assert cache.lens.tolist() == lens
        check_attention(o[rows], None, {"q": q[rows], "k_cache": cache.k[0], "ctx": [ctx[s] for s in seqs],
                                        "new": [new[s] for s in seqs], "keys": [hist[s][0] for s in seqs],
                                        "vals": [hist[s][1] for s in seqs]})
    assert lens[1] == 16
