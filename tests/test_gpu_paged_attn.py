"""Attention over a paged cache against 64-bit softmax: every mix of single tokens, drafted
tokens and chunks, at the sizes where tiles, pages and rows end inside one another."""
import ctypes
import math

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis
from paged_util import check_attention, make_batch
from paged_util import HALF_STEP

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def clean_error_word():
    clis.clis_clear_device_error()
    yield
    assert clis.clis_get_device_error() == 0


def run(b, causal=True, max_q=None, **kw):
    return clis.attention_paged(b["q"], b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], b["kv_len"],
                                b["max_q"] if max_q is None else max_q, causal=causal, return_lse=True, **kw)


# (ctx, new, H, Hkv, d, page, dtype, causal)
DECODE = [
    ([0], [1], 4, 4, 128, 16, BF, True),                       # one token, nothing cached before it
    ([1], [1], 8, 1, 64, 8, FP, True),
    ([15], [1], 4, 2, 128, 16, BF, True),                      # a page exactly full
    ([16], [1], 4, 2, 128, 16, FP, True),
    ([62, 63, 64, 65], [1, 1, 1, 1], 8, 2, 128, 64, BF, True),  # around one 64-key unit
    ([299], [1], 32, 8, 128, 16, BF, True),
    ([5000], [1], 32, 8, 128, 16, BF, True),                   # keys shared out over many blocks
    ([5000], [1], 5, 1, 64, 32, FP, True),
    ([100, 0, 7000, 31, 900], [1, 1, 1, 1, 1], 16, 4, 128, 16, FP, True),  # ragged
    ([100, 3, 700], [3, 0, 5], 12, 4, 64, 128, BF, True),      # drafted tokens, one sequence without any
    ([100, 3, 700], [4, 4, 4], 12, 4, 128, 8, BF, False),      # no mask among the new tokens
    ([2000, 10], [2, 2], 16, 1, 128, 256, BF, True),           # 32 rows
    ([513], [5], 6, 1, 128, 32, FP, True),                     # 30 rows
    ([40] * 40, [1] * 40, 6, 2, 64, 16, BF, True),             # more sequences than warps
]
CHUNK = [
    ([0], [33], 1, 1, 128, 16, BF, True),                      # one short prompt
    ([0], [128], 4, 4, 64, 64, FP, True),
    ([0], [129], 4, 2, 128, 128, BF, True),
    ([127], [257], 8, 2, 128, 8, FP, True),
    ([1000], [100], 8, 1, 128, 16, BF, True),
    ([1000], [100], 8, 1, 64, 16, BF, False),
    ([3000], [300], 5, 1, 128, 32, BF, True),                  # 25 tokens of 5 heads per row tile
    ([3000, 17], [40, 300], 3, 1, 64, 256, FP, True),          # 42 tokens of 3 heads
    ([500], [70], 128, 1, 128, 64, BF, True),                  # one token per row tile
    ([500], [40], 64, 1, 64, 64, BF, True),
    ([0, 300, 64, 0], [700, 1, 200, 65], 8, 4, 128, 16, BF, True),   # mixed
    ([900, 0, 20, 2000, 5], [1, 512, 0, 1, 300], 8, 2, 64, 32, FP, True),
    ([0], [2000], 16, 2, 128, 64, BF, True),                   # triangular costs
    ([127, 128, 129], [128, 128, 128], 2, 2, 128, 128, BF, False),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,d,page,dtype,causal", DECODE + CHUNK)
def test_against_64_bits(ctx, new, H, Hkv, d, page, dtype, causal):
    b = make_batch(ctx, new, H, Hkv, d, page, dtype, seed=len(ctx) + d + page)
    o, lse2 = run(b, causal)
    check_attention(o, lse2, b, causal)
    o2, lse3 = run(b, causal)
    assert torch.equal(o, o2) and torch.equal(lse2, lse3)  # reruns agree bit for bit


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ctx,new", [([700, 40], [1, 1]), ([300, 90], [150, 1])])
def test_strides(ctx, new, dtype):
    """q and o inside wider buffers and head-major, caches as [pages, page, H_kv, d]."""
    b = make_batch(ctx, new, 8, 2, 128, 32, dtype, seed=3, layout="nhd")
    want, _ = run(b)
    check_attention(want, None, b)
    T = b["q"].shape[0]
    wide = torch.randn(T, 12, 136, device="cuda").to(dtype)
    wide[:, 2:10, :128] = b["q"]
    out = torch.full((8, T, 128), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    got, _ = run({**b, "q": wide[:, 2:10, :128]}, out=out)
    assert got is out and torch.equal(got, want)
    head_major = b["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(run({**b, "q": head_major})[0], want)
    # heads that share one row of q (stride 0)
    shared = b["q"][:, :1].expand(-1, 8, -1)
    assert torch.equal(run({**b, "q": shared})[0], run({**b, "q": shared.contiguous()})[0])


@pytest.mark.parametrize("new", [[1, 2, 0], [1, 140, 0]])
def test_rows_of_no_sequence_stay(new):
    b = make_batch([50, 60, 70], new, 4, 2, 64, 16, BF, seed=5, extra_rows=37)
    T = b["q"].shape[0]
    out = torch.full((T, 4, 64), 3.0, dtype=BF, device="cuda")
    o, lse2 = run(b, out=out)
    check_attention(o, lse2, b)
    assert (o[sum(new):] == 3.0).all()


@pytest.mark.parametrize("max_q,H", [(1, 4), (64, 4)])
def test_rows_without_keys(max_q, H):
    """kv_len 0, and kv_len below the number of new tokens (its first tokens see nothing)."""
    for n, kv in ((1, 0), (max_q, 0), (max_q, max_q // 2)):
        b = make_batch([64], [n], H, 2, 128, 16, BF, seed=2)
        b["kv_len"] = torch.tensor([kv], dtype=torch.int32, device="cuda")
        o, lse2 = run(b)
        blind = n - kv
        assert (o[:blind] == 0).all() and (lse2[:blind] == -math.inf).all()
        if kv:
            seen = {**b, "ctx": [0], "new": [kv], "q": b["q"][blind:], "keys": [b["keys"][0][:kv]],
                    "vals": [b["vals"][0][:kv]]}
            check_attention(o[blind:], lse2[blind:], seen)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,new,H,Hkv,d", [([200], [4], 8, 2, 128), ([100], [90], 4, 1, 128), ([0], [300], 2, 2, 64),
                                             ([5000], [4], 4, 1, 64)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_masked_values_that_are_not_finite(bad, ctx, new, H, Hkv, d, dtype):
    """A key or value of a later token that is not finite reaches the rows that see it, and no other."""
    b = make_batch(ctx, new, H, Hkv, d, 16, dtype, seed=7)
    clean, clean_lse = run(b)
    at = ctx[0] + new[0] - 2          # the last token but one: seen by the last two
    page, row = b["block_table"][0, at // 16].item(), at % 16
    vc = b["v_cache"].clone()
    vc[page, :, row, 5] = bad
    o, lse2 = run({**b, "v_cache": vc})
    assert torch.equal(lse2, clean_lse)
    assert torch.equal(o[:-2], clean[:-2])
    rest = [c for c in range(d) if c != 5]
    assert torch.equal(o[-2:, :, rest], clean[-2:, :, rest])
    hit = o[-2:, :, 5].float()
    assert torch.isnan(hit).all() if math.isnan(bad) else (hit == bad).all()
    kc = b["k_cache"].clone()
    kc[page, :, row, 5] = float("nan")
    o, lse2 = run({**b, "k_cache": kc})
    assert torch.equal(o[:-2], clean[:-2]) and torch.isnan(o[-2:].float()).all() and torch.isnan(lse2[-2:]).all()


def test_a_key_that_is_not_finite_seen_by_all():
    """NaN keys make NaN rows, not rows without keys, also where a whole tile is NaN."""
    for new in ([1], [40]):
        b = make_batch([300], new, 4, 2, 128, 16, BF, seed=11)
        b["k_cache"][b["block_table"][0, :16].long()] = float("nan")  # the first 256 keys
        o, lse2 = run(b)
        assert torch.isnan(o.float()).all() and torch.isnan(lse2).all()


def test_many_sequences():
    """More sequences than threads of the kernels that list the work."""
    new = [1 if i % 3 else 0 for i in range(1100)]
    b = make_batch([(7 * i) % 90 for i in range(1100)], new, 4, 2, 64, 8, BF, seed=37)
    check_attention(*run(b), b, what="single tokens")
    new[550] = 40
    new[1099] = 33
    b = make_batch([(7 * i) % 90 for i in range(1100)], new, 4, 2, 64, 8, BF, seed=38)
    check_attention(*run(b), b, what="with chunks")


def test_the_most_sequences():
    """16,384 sequences, nearly all of them without a token in this step."""
    ctx, new = [0] * 16384, [0] * 16384
    for s, c, n in ((0, 100, 1), (7, 0, 1), (511, 300, 60), (9000, 64, 1), (16383, 33, 2)):
        ctx[s], new[s] = c, n
    b = make_batch(ctx, new, 4, 2, 64, 16, BF, seed=39)
    check_attention(*run(b), b)
    new[511] = 1
    b = make_batch(ctx, new, 4, 2, 64, 16, BF, seed=40)
    check_attention(*run(b), b)


def test_calls_at_once():
    """Calls on several streams at the same time, each with its own workspace."""
    bs = [make_batch([900, 40], [1, n], 8, 2, 128, 16, BF, seed=50 + i) for i, n in enumerate((1, 90, 3, 200))]
    want = [run(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for b, s in zip(bs, streams):
            with torch.cuda.stream(s):
                got.append(run(b))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1])


@pytest.mark.parametrize("Hkv,g,n,ctx,dtype", [(8, 4, 640, 8000, BF), (4, 2, 1200, 5000, FP), (1, 8, 60, 30000, BF),
                                               (2, 4, 500, 20000, BF), (16, 8, 16, 3000, BF), (8, 4, 9, 60000, FP)])
def test_parts_join_alike_whoever_is_last(Hkv, g, n, ctx, dtype):
    """Items as long as one to many blocks' runs: their parts end at about the same time, and reruns
    agree bit for bit whichever block joins them."""
    b = make_batch([ctx], [n], Hkv * g, Hkv, 128, 64, dtype, seed=41)
    o, lse2 = run(b)
    check_attention(o, lse2, b)
    for _ in range(20):
        o2, l2 = run(b)
        assert torch.equal(o, o2) and torch.equal(lse2, l2)


def test_sizes_of_one_with_odd_strides():
    """Dimensions of size 1 whose strides are not multiples of anything (torch leaves them as they are)."""
    b = make_batch([37], [1], 2, 1, 64, 16, BF, seed=43)
    want, _ = run(b)
    q = torch.empty(7 + 128, dtype=BF, device="cuda")[:128].as_strided((1, 2, 64), (3, 64, 1))
    q.copy_(b["q"])
    kc = b["k_cache"].as_strided(b["k_cache"].shape, (b["k_cache"].stride(0), 5, 64, 1))
    vc = b["v_cache"].as_strided(b["v_cache"].shape, (b["v_cache"].stride(0), 1, 64, 1))
    got, _ = run({**b, "q": q, "k_cache": kc, "v_cache": vc})
    assert torch.equal(got, want)


def test_max_q_only_chooses_the_kernel():
    """The decode kernel's and the chunk kernel's results agree to rounding; T is always a valid max_q."""
    b = make_batch([300, 900, 64], [1, 2, 1], 8, 2, 128, 16, BF, seed=13)
    for mq in (2, 4, 100, 10 ** 9):
        check_attention(*run(b, max_q=mq), b, what=f"max_q {mq}")


def test_large_scores_raise_the_shift_often():
    """Scores that grow along the keys: the running shift is raised again and again."""
    for new in ([1], [100]):
        b = make_batch([1500], new, 4, 1, 128, 32, BF, seed=17)
        n = 1500 + new[0]
        ramp = torch.linspace(0.05, 3.0, n, device="cuda")[:, None, None]
        # keys along one direction, longer and longer; queries along the same direction
        e = torch.zeros(128, device="cuda")
        e[:8] = 1.0
        keys = (ramp * e).to(BF)
        b["keys"] = [keys]
        for i in range(-(-n // 32)):
            m = min(32, n - 32 * i)
            b["k_cache"][b["block_table"][0, i].item(), :, :m] = keys[32 * i:32 * i + m].transpose(0, 1)
        b["q"] = (10 * e).to(BF).expand(new[0], 4, 128).contiguous()
        o, lse2 = run(b)
        check_attention(o, lse2, b)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the page offset needs 64 bits."""
    pages, page, d = 70000, 256, 128
    kc = torch.empty((pages, 2, page, d), dtype=BF, device="cuda")  # 4.6e9 elements, 9.2 GB
    vc = torch.empty_like(kc)
    for new in ([1], [80]):
        n = 600 + new[0]
        b = make_batch([600], new, 4, 2, d, page, BF, seed=19, poison=False)
        ids = [pages - 1, pages - 7, 40000]
        for i, p in enumerate(ids):
            src = b["block_table"][0, i].item()
            kc[p], vc[p] = b["k_cache"][src], b["v_cache"][src]
        b["block_table"][0, :3] = torch.tensor(ids, dtype=torch.int32)
        check_attention(*run({**b, "k_cache": kc, "v_cache": vc}), b)
        assert n <= 3 * page


def test_other_stream_and_captured_graph():
    """A captured call replayed with other lengths; two graphs with workspaces of their own."""
    b = make_batch([700, 300], [1, 1], 8, 2, 128, 16, BF, seed=23)
    c = make_batch([40, 500], [90, 1], 8, 2, 128, 16, BF, seed=24)
    want = [run(x) for x in (b, c)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [run(x) for x in (b, c)]
    torch.cuda.current_stream().wait_stream(side)
    for (o, l), (o2, l2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(l, l2)
    graphs = []
    for x in (b, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = run(x)
        graphs.append((g, r))
    for (g, r), w in zip(graphs, want):
        r[0].zero_()
    for g, r in graphs:
        g.replay()
    torch.cuda.synchronize()
    for (g, r), w in zip(graphs, want):
        assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])
    # other lengths in the same buffers
    b["kv_len"].copy_(torch.tensor([333, 17], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    short = {**b, "ctx": [332, 16], "keys": [b["keys"][0][:333], b["keys"][1][:17]],
             "vals": [b["vals"][0][:333], b["vals"][1][:17]]}
    check_attention(*graphs[0][1], short)


def test_bad_pages_and_lengths_are_recorded():
    for new in ([2], [80]):
        b = make_batch([100], new, 4, 2, 128, 16, BF, seed=29)
        b["block_table"][0, 1] = b["k_cache"].shape[0]      # one page out of range: zeros
        o, _ = run(b)
        assert torch.isfinite(o.float()).all()
        assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
        clis.clis_clear_device_error()
        zero = {**b, "keys": [b["keys"][0].clone()], "vals": [b["vals"][0].clone()]}
        zero["keys"][0][16:32] = 0
        zero["vals"][0][16:32] = 0
        check_attention(o, None, zero)
        b["block_table"][0, 1] = -5
        run(b)
        assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
        clis.clis_clear_device_error()
        # a length beyond the block table, prefix sums beyond T: brought into range
        b = make_batch([100], new, 4, 2, 128, 16, BF, seed=29, poison=False)
        b["block_table"].clamp_(min=0)
        b["kv_len"].fill_(10 ** 9)
        b["cu_q"][1] = 10 ** 6
        run(b)
        assert clis.clis_get_device_error() & clis.PAGED_LENGTH_BIT
        clis.clis_clear_device_error()


def test_more_tokens_than_max_q_is_recorded():
    b = make_batch([10, 10], [1, 9], 4, 1, 64, 16, BF, seed=31)
    run(b, max_q=4)
    assert clis.clis_get_device_error() == clis.PAGED_LENGTH_BIT
    clis.clis_clear_device_error()


def test_empty_batches():
    b = make_batch([10], [1], 4, 2, 64, 16, BF, seed=1)
    o = clis.attention_paged(b["q"][:0], b["k_cache"], b["v_cache"], b["block_table"], torch.zeros(2, dtype=torch.int32, device="cuda"),
                             b["kv_len"])
    assert o.shape == (0, 4, 64)
    none = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    out = torch.full((1, 4, 64), 2.0, dtype=BF, device="cuda")
    clis.attention_paged(b["q"], b["k_cache"], b["v_cache"], none, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         none[:, 0].contiguous(), out=out)
    assert (out == 2.0).all()


def test_prefix_sums_that_fall_stay_inside_the_workspace():
    """Sequences that share rows make more work items than T rows can: what is beyond the list is left out and
    recorded, nothing behind the workspace is touched, and a sound call afterwards is what it was."""
    S, T, H, Hkv, d = 64, 2048, 32, 8, 64
    b = make_batch([0], [T], H, Hkv, d, 64, BF, seed=61)
    want, want_lse = run(b)
    desc = clis.PagedDesc(S=S, T=T, H=H, Hkv=Hkv, d=d, page_size=64, num_pages=b["k_cache"].shape[0], width=b["block_table"].shape[1],
                          q_st=H * d, q_sh=d, o_st=H * d, o_sh=d, kc_sp=Hkv * 64 * d, kc_sh=64 * d, kc_sn=d, vc_sp=Hkv * 64 * d,
                          vc_sh=64 * d, vc_sn=d, bt_ss=b["block_table"].shape[1], dtype=0)
    need = ctypes.c_size_t()
    assert clis.load_library().clis_attn_paged_workspace_size(desc, T, ctypes.byref(need)) == 0
    ws = torch.full((need.value + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([T * (s % 2) for s in range(S + 1)], dtype=torch.int32, device="cuda")
    kv = torch.full((S,), 90, dtype=torch.int32, device="cuda")
    bt = b["block_table"][:, :].expand(S, -1).contiguous()
    clis.clis_attn_fwd_paged(b["q"], b["k_cache"], b["v_cache"], bt, cu, kv, T, clis.scale_log2_for(d), workspace=ws)
    assert clis.clis_get_device_error() == clis.PAGED_LENGTH_BIT
    clis.clis_clear_device_error()
    assert (ws[need.value:] == 0x5A).all()
    o, lse2 = run(b)
    assert torch.equal(o, want) and torch.equal(lse2, want_lse)


@pytest.mark.parametrize("entry", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("new", [[2], [80]])
def test_any_page_number_out_of_range_reads_as_zeros(new, entry):
    """Whatever the block table holds for a visible key, a number that is no page is recorded and its keys and
    values are zeros (in the ring of the chunk kernel the tile before has left others)."""
    b = make_batch([300], new, 4, 2, 128, 16, BF, seed=29)
    b["block_table"][0, 11] = entry
    o, lse2 = run(b)
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
    clis.clis_clear_device_error()
    b["keys"][0][176:192] = 0
    b["vals"][0][176:192] = 0
    check_attention(o, lse2, b)


def test_a_long_run_without_edge_tiles():
    """Seconds of keys in whole tiles (no row has a masked place among them) before the last sequence's odd length:
    no wait of the kernel spans more than one work item.  All block tables name one page 64 times over."""
    S, n, g, Hkv, d, page, times = 332, 64, 4, 32, 64, 65536, 64
    gen = torch.Generator(device="cuda").manual_seed(71)
    kc, vc = (torch.randn((1, Hkv, page, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((S * n, g * Hkv, d), generator=gen, device="cuda").to(BF)
    bt = torch.zeros(S, times, dtype=torch.int32, device="cuda")
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    kv = torch.full((S,), page * times, dtype=torch.int32, device="cuda")
    kv[-1] -= 1
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    o, lse2 = clis.attention_paged(q, kc, vc, bt, cu, kv, n, causal=False, return_lse=True)
    end.record()
    torch.cuda.synchronize()
    assert clis.clis_get_device_error() == 0
    print(f"{start.elapsed_time(end) / 1e3:.2f} s")
    count = torch.full((page,), float(times), dtype=torch.float64, device="cuda")
    u = HALF_STEP[BF]
    for s in (0, S - 1):
        if s:
            count[-1] -= 1
        for h in (0, Hkv - 1):
            rows, heads = slice(s * n, s * n + n), slice(h * g, h * g + g)
            x = q[rows, heads].double() @ kc[0, h].double().T / 8.0
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - m) * count
            L = p.sum(-1, keepdim=True)
            want, A = p @ vc[0, h].double() / L, p @ vc[0, h].double().abs() / L
            # as check_attention, and 32-bit sums over 2^15 key tiles: 2^-24 each of a row sum, 2^-23 of an output in each
            # of a tile's eight products (whose sum may be cut off instead of rounded)
            tol = u * (want.abs() + A) * 1.01 + 2e-4 * A + want.abs() * (2.0 ** 15 * 2.0 ** -24 + 2.0 ** 18 * 2.0 ** -23)
            assert ((o[rows, heads].double() - want).abs() <= tol).all(), (s, h)
            e = (lse2[rows, heads].double() - (m + L.log())[..., 0] / math.log(2.0)).abs().max().item()
            assert e <= 1.5e-4 + 2.0 ** 15 * 2.0 ** -24 / math.log(2.0) + 2.0 ** -23 * 30, (s, h, e)


def test_the_largest_table():
    """16,384 sequences whose table rows could hold 2^26 keys each, with 8 key/value heads; they hold a few."""
    S, Hkv, d, page = 16384, 8, 64, 65536
    g = torch.Generator(device="cuda").manual_seed(73)
    kc, vc = (torch.randn((2, Hkv, page, d), generator=g, device="cuda").to(BF) for _ in range(2))
    bt = torch.full((S, 1024), 0x3FFFFFFF, dtype=torch.int32, device="cuda")
    bt[:, 0] = torch.arange(S, device="cuda") % 2
    for n in (1, 3):                      # single tokens; few sequences with chunks among them
        new = torch.ones(S, dtype=torch.int64) if n == 1 else torch.zeros(S, dtype=torch.int64)
        if n > 1:
            new[[5, 700, 16383]] = torch.tensor([40, 1, 130])
        cu = torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0))).to(torch.int32).cuda()
        kv = (torch.arange(S) % 37 + new).to(torch.int32).cuda()
        T = int(new.sum())
        q = torch.randn((T, Hkv, d), generator=g, device="cuda").to(BF)
        o, lse2 = clis.attention_paged(q, kc, vc, bt, cu, kv, int(new.max()), return_lse=True)
        for s in (0, 1, 5, 36, 700, 8191, 16382, 16383):
            r, m, c = cu[s].item(), int(new[s]), s % 37
            if m == 0:
                continue
            check_attention(o[r:r + m], lse2[r:r + m], {"q": q[r:r + m], "k_cache": kc, "ctx": [c], "new": [m],
                                                       "keys": [kc[s % 2, :, :c + m].transpose(0, 1)],
                                                       "vals": [vc[s % 2, :, :c + m].transpose(0, 1)]})


@pytest.mark.parametrize("S,n,H", [(1300, 1, 1), (320, 40, 4)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_small_weights_beside_a_large_one(S, n, H, dtype):
    """One key far above 262,143 others, whose weights are 2^-25.5 of its own each: together 0.6%.  Enough sequences
    that none is shared out, so that all of a row's weights are taken with one shift."""
    d, page, N = 64, 65536, 262144
    kc, vc = torch.zeros(4, 1, page, d, dtype=dtype, device="cuda"), torch.ones(4, 1, page, d, dtype=dtype, device="cuda")
    q = torch.zeros(S * n, H, d, dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    kc[0, 0, 0, 0] = 17.625
    vc[0, 0, 0] = 0.0
    bt = torch.arange(4, dtype=torch.int32, device="cuda").expand(S, 4).contiguous()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    kv = torch.full((S,), N, dtype=torch.int32, device="cuda")
    o = clis.attention_paged(q, kc, vc, bt, cu, kv, n, causal=False)
    top = 8.0 * 17.625 / 8.0 / math.log(2.0)
    L = 1.0 + (N - 1) * 2.0 ** -top
    want = (N - 1) * 2.0 ** -top / L
    u = HALF_STEP[dtype]
    # as check_attention, with A = o here; weights below 2^-14 of 2^7 times the largest lose up to 2^-25: 2^-32 of it each
    tol = 2 * u * want * 1.01 + 2e-4 * want + ((N - 1) / L * 2.0 ** -32 + 2.0 ** -25 if dtype == FP else 0)
    err = (o.double() - want).abs().max().item()
    assert err <= tol, f"off by {err:.2e} of {want:.2e}, {err / tol:.1f} times the bound"


@pytest.mark.parametrize("S,n,H", [(1300, 1, 1), (320, 40, 4)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_row_sums_of_many_small_weights(S, n, H, dtype, d):
    """262,143 weights of 2^-25.5 beside one of 1 are 0.008 of lse2, and more than the weights' own steps:
    32-bit sums that add them one unit at a time must not lose them."""
    page, N = 65536, 262144
    kc = torch.zeros(4, 1, page, d, dtype=dtype, device="cuda")
    q = torch.zeros(S * n, H, d, dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    kc[0, 0, 0, 0] = 17.625
    bt = torch.arange(4, dtype=torch.int32, device="cuda").expand(S, 4).contiguous()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    kv = torch.full((S,), N, dtype=torch.int32, device="cuda")
    _, lse2 = clis.attention_paged(q, kc, kc, bt, cu, kv, n, softmax_scale=0.125, causal=False, return_lse=True)
    top = 8.0 * 17.625 / 8.0 / math.log(2.0)
    want = top + math.log2(1.0 + (N - 1) * 2.0 ** -top)
    # as check_attention; the chunk kernel adds a key tile's sum at a time: half a step of the row sum each
    tol = 1.5e-4 + 2.0 ** -23 * top + (N / 128 * 2.0 ** -24 / math.log(2.0) if n > 1 else 0)
    err = (lse2.double() - want).abs().max().item()
    assert err <= tol, f"off by {err:.2e}, {err / tol:.1f} times the bound"


@pytest.mark.parametrize("scale", [1.0, 0.02, 0.37])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)])
def test_softmax_scales(scale, dtype, d):
    """Scales other than 1 / sqrt(d), single tokens and chunks; large ones make one weight of a row stand out."""
    for new in ([1, 2, 1], [1, 130, 0]):
        b = make_batch([300, 70, 900], new, 8, 2, d, 32, dtype, seed=81)
        b["q"] = (b["q"].float() * (1.0 / (8.0 * scale))).to(dtype)   # scores of the usual size, which the bounds are for
        o, lse2 = run(b, softmax_scale=scale)
        check_attention(o, lse2, b, scale=scale)


@pytest.mark.parametrize("page", [512, 4096, 65536])
@pytest.mark.parametrize("new", [[1, 3], [200, 1]])
def test_large_pages(page, new):
    b = make_batch([700, page + 100], new, 4, 2, 128, page, BF, seed=83)
    check_attention(*run(b), b)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_the_longest_sequence(n, dtype):
    """2^26 - 3 keys (one page, 1,024 times over) in one sequence, shared out over the whole GPU."""
    page, times, d = 65536, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(85)
    kc, vc = (torch.randn((1, 1, page, d), generator=gen, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((n, 4, d), generator=gen, device="cuda").to(dtype)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    o, lse2 = clis.attention_paged(q, kc, vc, torch.zeros(1, times, dtype=torch.int32, device="cuda"), i32([0, n]),
                                   i32([page * times - 3]), n, causal=True, return_lse=True)
    count = torch.full((n, page), float(times), dtype=torch.float64, device="cuda")
    for i in range(n):                                  # query i is key 2^26 - 3 - n + i
        count[i, page - 3 - n + i + 1:] -= 1
    x = q.double().transpose(0, 1) @ kc[0, 0].double().T / 8.0
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m) * count
    L = p.sum(-1, keepdim=True)
    v = vc[0, 0].double()
    want, A = ((p @ t / L).transpose(0, 1) for t in (v, v.abs()))
    u = HALF_STEP[dtype]
    # as check_attention; 32-bit sums: a run is at most 2^26 / 152 keys, 16 to a product, each of which may cut off 2^-23
    tol = u * (want.abs() + A) * 1.01 + 2e-4 * A + want.abs() * (2.0 ** 26 / 152 / 16 * 2.0 ** -23) + 2.0 ** -25
    assert ((o.double() - want).abs() <= tol).all()
    e = (lse2.double() - ((m + L.log())[..., 0] / math.log(2.0)).transpose(0, 1)).abs().max().item()
    assert e <= 1.5e-4 + 2.0 ** -23 * 32 + 2.0 ** 26 / 152 / 128 * 2.0 ** -24 / math.log(2.0), e
