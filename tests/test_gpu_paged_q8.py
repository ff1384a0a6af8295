"""A paged cache held in 8 bits: the quantising write, reading back, and attention over the codes."""
import math

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis
from q8_util import CODES, TOP, check_q8, few_rows, make_q8, raw

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _clean():
    clis.clis_clear_device_error()
    yield
    torch.cuda.synchronize()
    assert clis.clis_get_device_error() == 0


def attend(b, **kw):
    return clis.attention_paged(b["q"], b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], b["kv_len"],
                                kw.pop("max_q", b["max_q"]), k_scale=b["k_scale"], v_scale=b["v_scale"], **kw)


# ------------------------------------------------------------------ attention

SHAPES = [  # ctx, new, H, Hkv, d, page
    ([0], [1], 1, 1, 128, 8),                                   # one key
    ([300], [1], 32, 8, 128, 16),
    ([31, 32, 33, 0, 95, 1000], [1] * 6, 8, 8, 128, 16),        # around a unit's 32 keys
    ([63, 64, 65, 0, 127, 1000], [1] * 6, 8, 2, 64, 32),        # and 64 at d = 64
    ([700, 0, 5, 2000], [1, 0, 1, 1], 12, 4, 64, 8),            # a sequence without a token
    ([500, 3, 90], [5, 2, 0], 16, 4, 128, 64),                  # drafted tokens: 20 rows
    ([500, 3, 90, 1500], [5, 1, 4, 5], 32, 4, 128, 16),         # 40 rows
    ([77, 1200], [13, 16], 16, 4, 64, 128),                     # 64 rows
    ([40, 0], [2, 3], 128, 8, 128, 8),                          # 16 heads a key: 48 rows
    ([10], [1], 128, 1, 64, 16),                                # 128 query heads a key
    ([200, 0, 33], [70, 129, 1], 8, 2, 128, 16),                # small chunks and a single token: 516 rows
    ([200, 5, 300, 17], [17, 300, 1, 2], 4, 4, 64, 8),
    ([4000], [9], 40, 8, 128, 256),
    # the same with tables that can hold far more: the chunk kernel
    ([10], [1], 128, 1, 64, 16, 30000),
    ([200, 0, 33], [70, 129, 1], 8, 2, 128, 16, 20000),
    ([200, 5, 300, 17], [17, 300, 1, 2], 4, 4, 64, 8, 30000),
    ([4000, 70], [20, 1], 40, 8, 128, 256, 1000),
    ([300, 20], [600, 1], 16, 4, 128, 32),                      # 2,400 rows: the chunk kernel for the single token too
    ([500, 3, 90, 3000], [3, 1, 2, 3], 32, 4, 64, 16),          # 24 rows at d = 64
    ([500, 3, 900], [3, 0, 7], 8, 2, 64, 8),                    # 28 rows
    ([2500, 64, 1], [10, 7, 1], 20, 4, 64, 64),                 # 50 rows
]


def which(b):
    """The kernels that the batch's sequences run."""
    g = b["q"].shape[1] // b["k_cache"].shape[1]
    return {"few" if n * g <= few_rows(b) else "chunk" for n in b["new"] if n}


def test_the_shapes_cover_the_ways():
    ways = [which(make_q8(*s[:6], BF, "int8", columns=s[6] if len(s) > 6 else 0)) for s in SHAPES]
    assert {"few"} in ways and {"chunk"} in ways and {"few", "chunk"} in ways


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,code", [(BF, "int8"), (HF, "int8"), (BF, "e4m3"), (HF, "e4m3")])
def test_attention(shape, dtype, code):
    ctx, new, H, Hkv, d, page, *columns = SHAPES[shape]
    b = make_q8(ctx, new, H, Hkv, d, page, dtype, code, seed=shape, extra_rows=2, layout="hnd" if shape % 2 else "nhd", columns=sum(columns))
    causal = shape % 3 != 2
    out = torch.full_like(b["q"], 7.0)
    o, lse = attend(b, causal=causal, out=out, return_lse=True)
    check_q8(o, lse, b, causal, what=f"{SHAPES[shape]}")
    assert (o[sum(new):] == 7.0).all()  # rows of no sequence


@pytest.mark.parametrize("shape", [i for i, s in enumerate(SHAPES) if len(s) == 6 and max(s[1]) * s[2] // s[3] <= 64])
@pytest.mark.parametrize("dtype,code", [(BF, "int8"), (HF, "e4m3")])
def test_short_sequences_in_long_tables(shape, dtype, code):
    """Few rows: with short tables a block takes an item, with long ones runs of units are joined by a second launch."""
    ctx, new, H, Hkv, d, page = SHAPES[shape]
    b = make_q8(ctx, new, H, Hkv, d, page, dtype, code, seed=100 + shape, columns=4096 // page)
    o, lse = attend(b, return_lse=True)
    check_q8(o, lse, b, what=f"{SHAPES[shape]}")
    short = dict(b, block_table=b["block_table"][:, :-4096 // page].contiguous())
    o, lse = attend(short, return_lse=True)
    check_q8(o, lse, short, what=f"{SHAPES[shape]}, short tables")


@pytest.mark.parametrize("d,ctx", [(128, 127), (128, 1000), (64, 1000), (64, 2040)])
@pytest.mark.parametrize("new", [1, 2, 5])
def test_sixty_four_items_of_up_to_32_units(d, ctx, new):
    b = make_q8([ctx - 7 * i for i in range(16)], [new] * 16, 16, 4, d, 8, BF, "int8", seed=ctx + new)
    check_q8(attend(b), None, b)


@pytest.mark.parametrize("dtype,code", [(BF, "int8"), (HF, "e4m3")])
def test_blocks_of_single_tokens_beside_a_chunk(dtype, code):
    """Tables of fewer than 32 units but more than 16 MB of codes: a block per item between unpacking and the chunk kernel."""
    b = make_q8([900 - 13 * i for i in range(47)] + [600], [1] * 47 + [300], 32, 8, 128, 16, dtype, code, seed=48)
    assert which(b) == {"few", "chunk"}
    o, lse = attend(b, return_lse=True)
    check_q8(o, lse, b)
    assert torch.equal(attend(b), o)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("new,H", [([1] * 9, 8), ([4, 1, 3, 2, 4, 1, 1, 4, 2], 16)])
def test_many_lengths_and_joins(code, new, H):
    ctx = [1, 5000, 17, 900, 0, 12000, 333, 64, 2047]
    b = make_q8(ctx, new, H, 2, 128, 32, BF, code, seed=3)
    o, lse = attend(b, return_lse=True)
    check_q8(o, lse, b)
    assert torch.equal(o, attend(b))  # reruns agree bit for bit


def test_hundreds_of_sequences():
    ctx = [(37 * i) % 211 for i in range(700)]
    b = make_q8(ctx, [1] * 700, 8, 4, 64, 16, HF, "int8", seed=5)
    check_q8(attend(b), None, b)


@pytest.mark.parametrize("spread", [4.0, 12.0])
@pytest.mark.parametrize("new", [[1, 1], [3, 2]])
def test_scales_of_any_size(spread, new):
    """V's scales span many powers of two (log2: 4 * 1.44 * 3 each way, or 50), K's are ordinary."""
    b = make_q8([800, 50], new, 8, 2, 128, 16, BF, "int8", seed=7)
    g = torch.Generator(device="cuda").manual_seed(1)
    for s in range(2):
        (kc, ks), (vc, vs) = b["keys"][s]
        vs *= torch.exp(spread * torch.randn(vs.shape, generator=g, device="cuda"))
        b["keys"][s] = [(kc, ks), (vc, vs)]
        for i in range(vs.shape[0]):
            b["v_scale"][b["block_table"][s, i // 16], :, i % 16] = vs[i]
    check_q8(attend(b), None, b)


def scaled(b, q=1.0, k=1.0):
    """The batch with its rows of q times `q` (a number, or one per row and head) and K's scales times `k`."""
    b["q"] = (b["q"].float() * q).to(b["q"].dtype)
    b["k_scale"] = b["k_scale"] * k
    b["keys"] = [[(kc, ks * k), v] for (kc, ks), v in b["keys"]]
    return b


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [-112, -60, 60, 112])
@pytest.mark.parametrize("new,H,d,columns", [(1, 4, 128, 0), (5, 16, 128, 0), (6, 8, 64, 0), (90, 4, 128, 0), (90, 4, 128, 20000)])
def test_key_scales_of_any_size(new, H, d, columns, power, code):
    """Keys far larger or smaller than ordinary ones and queries the other way round: the scores are the ordinary ones."""
    b = make_q8([900, 40], [new, 1], H, 2, d, 16, BF, code, seed=3, columns=columns)
    check_q8(*attend(scaled(b, 2.0 ** -power, 2.0 ** power), return_lse=True), b)


@pytest.mark.parametrize("d,new", [(128, 1), (128, 4), (64, 6)])
def test_query_rows_of_different_sizes(d, new):
    """Some heads' queries are 2^-112, 2^-115 or zero, and K's scales 2^112; a head of ordinary numbers among them, whose scores
    are beyond any sense, changes nothing for the others."""
    b = make_q8([300, 40], [new, 1], 8, 2, d, 16, BF, "int8", seed=4)
    size = torch.full((new + 1, 8, 1), 2.0 ** -112, device="cuda")
    size[:, 1] = 0.0
    size[:, 5] = 2.0 ** -115
    size[:, 6] = 0.0
    q = b["q"]
    o, lse = attend(scaled(b, size, 2.0 ** 112), return_lse=True)
    check_q8(o, lse, b)
    b["q"] = b["q"].clone()
    b["q"][:, 1] = q[:, 1]
    o2, lse2 = attend(b, return_lse=True)
    others = [h for h in range(8) if h != 1]
    assert torch.equal(o[:, others], o2[:, others]) and torch.equal(lse[:, others], lse2[:, others])


@pytest.mark.parametrize("H,new,d", [(8, 1, 64), (8, 1, 128), (32, 2, 128)])
@pytest.mark.parametrize("power", [-107, 0, 100])
def test_many_small_weights_of_values_of_any_size(H, new, d, power):
    """One key with a weight of 1 and 30,000 with 2^-20 each, together 3% of a row: they count whatever V's scales are, down to
    those of the smallest rows that a write keeps (2^-100 over 127).  400 requests of the same pages, so that the runs are long."""
    N, S = 30000, 400
    b = make_q8([N], [new], H, 4, d, 64, BF, "int8", seed=6)
    (kc, ks), (vc, vs) = b["keys"][0]
    kc.zero_()
    kc[7, :, 3] = 127
    ks.fill_(1.0)
    vc.abs_().clamp_(min=20)
    vc[7] = -vc[7]
    vs.fill_(2.0 ** power)
    at = torch.arange(N + new, device="cuda")
    pages = b["block_table"][0].long()[at // 64]
    for cache, scale, (c, x) in ((b["k_cache"], b["k_scale"], (kc, ks)), (b["v_cache"], b["v_scale"], (vc, vs))):
        cache[pages, :, at % 64] = c
        scale[pages, :, at % 64] = x
    b["q"].zero_()
    b["q"][:, :, 3] = 1.0
    many = dict(b, q=b["q"].repeat(S, 1, 1), block_table=b["block_table"].repeat(S, 1), kv_len=b["kv_len"].repeat(S),
                cu_q=torch.arange(0, new * S + 1, new, dtype=torch.int32, device="cuda"))
    softmax_scale = 20 * math.log(2) / 127
    o, lse = attend(many, softmax_scale=softmax_scale, return_lse=True)
    one = dict(b, keys=[[(kc, ks), (vc, torch.ones_like(vs))]])
    for r in range(0, new * S, new * 57):
        check_q8(o[r:r + new].double() * 2.0 ** -power, lse[r:r + new], one, scale=softmax_scale)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("power,columns", [(-102, 0), (-102, 300), (125, 0), (125, 300)])
@pytest.mark.parametrize("new,H,d", [(1, 4, 128), (3, 12, 64)])
def test_values_of_any_size(new, H, d, power, columns, code):
    """V's rows near the smallest that a write keeps and near bf16's largest numbers (three keys: their sum must fit 32 bits)."""
    b = make_q8([2, 1], [new, 1], H, 2, d, 16, BF, code, seed=9, columns=columns, spread=0.0)
    b["v_scale"] = b["v_scale"] * 2.0 ** power
    o = attend(b)
    check_q8(o.double() * 2.0 ** -power, None, b)


@pytest.mark.parametrize("H", [2, 12])
def test_fp16_queries_are_exact(H):
    """Rows of fp16 with its largest and its smallest numbers: what the small ones add to a score is not rounded."""
    b = make_q8([0], [1], H, 1, 64, 8, HF, "int8", seed=8)
    (kc, ks), _ = b["keys"][0]
    kc.fill_(101)
    kc[..., 0] = 0
    ks.fill_(2.0 ** 12)
    b["k_cache"][b["block_table"][0, 0], :, 0] = kc[0]
    b["k_scale"][b["block_table"][0, 0], :, 0] = 2.0 ** 12
    b["q"][:] = (2 * torch.arange(64, device="cuda") + 1) * 2.0 ** -24   # (odd multiples of the smallest number)
    b["q"][..., 0] = 60000.0
    _, lse = attend(b, softmax_scale=1.0, return_lse=True)
    want = (b["q"][0].double() * kc[0, 0].double()).sum(-1) * 2.0 ** 12 / math.log(2)
    # a product is exact, their sum rounded in 32 bits: 64 additions; then two factors, one of them rounded itself
    assert ((lse[0].double() - want).abs() <= 67 * 2.0 ** -24 * want).all()


def test_chunk_with_scales_of_zero_and_of_any_size():
    """K's scales of 0, 2^-110, 2^-60 and 2^20 among a chunk's: scores of no and of great size."""
    b = make_q8([300, 11], [70, 90], 4, 2, 64, 8, BF, "e4m3", seed=15, columns=50000)
    assert which(b) == {"chunk"}
    (kc, ks), (vc, vs) = b["keys"][0]
    for i, x in ((3, 0.0), (50, 2.0 ** -110), (120, 2.0 ** -60), (310, 0.0), (330, 2.0 ** -110)):
        ks[i] = x
        b["k_scale"][b["block_table"][0, i // 8], :, i % 8] = x
    check_q8(attend(b), None, b)
    b["k_scale"][b["block_table"][0, 4].long(), 1, 3] = 2.0 ** 20  # key 35 of the second head takes all or nothing
    o = attend(b)
    assert torch.isfinite(o).all()
    sign = (b["q"][:70, 2:].double() @ kc[35, 1].float().double()) > 0
    v = (vc[35, 1].float() * vs[35, 1]).to(BF)
    # Weight 2^e of one key, e the rounding of its score (up to half a step of 2^28, not 0): rounded to bf16 for the
    # product, not for the row sum, and the output is rounded: two half steps.
    assert ((o[:70, 2:][sign].double() - v.double()).abs() <= 2.0 ** -7 * 1.01 * v.double().abs()).all()


def test_zero_scales_and_rows():
    b = make_q8([40, 3], [1, 1], 4, 2, 64, 16, BF, "int8", seed=8)
    for t in (b["v_scale"], b["k_scale"]):
        t[b["block_table"][1, 0]] = 0.0
    for s in ("v_scale",):
        b[s][b["block_table"][0, 0].long(), :, :5] = 0.0
    o = attend(b)
    assert (o[1] == 0).all() and torch.isfinite(o).all()
    (kc, ks), (vc, vs) = b["keys"][0]
    vs[:5] = 0.0
    b["keys"] = b["keys"][:1]
    b["ctx"], b["new"] = [40], [1]
    check_q8(o, None, b)


def test_no_keys():
    b = make_q8([5, 6], [1, 2], 4, 2, 128, 16, BF, "e4m3", seed=9)
    b["kv_len"].zero_()
    o, lse = attend(b, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("what", ["k_scale", "v_scale", "v_inf", "k_code", "v_code"])
@pytest.mark.parametrize("new,H,columns", [(3, 4, 0), (5, 16, 0), (40, 4, 0), (40, 4, 20000)])
def test_non_finite_where_some_rows_do_not_see_it(code, what, new, H, columns):
    """The last new token's key is no number: earlier rows are as without it, the last row is NaN."""
    if what.endswith("code") and code == "int8":
        pytest.skip("int8 codes are numbers")
    b = make_q8([61, 30], [new, new], H, 2, 64, 16, BF, code, seed=10, columns=columns)
    assert which(b) == {"chunk" if columns else "few"}
    want = attend(b)
    at = 61 + new - 1
    page, row = b["block_table"][0, at // 16].long(), at % 16
    if what.endswith("scale"):
        b[what][page, :, row] = math.nan
    elif what == "v_inf":
        b["v_scale"][page, :, row] = math.inf
    else:
        raw(b["k_cache" if what == "k_code" else "v_cache"])[page, :, row, ::3] = 127
    got = attend(b)
    assert torch.equal(got[:new - 1], want[:new - 1]) and torch.equal(got[new:], want[new:])
    last = got[new - 1]
    if what == "v_code":
        assert torch.isnan(last[:, ::3]).all()
        rest = torch.ones(64, dtype=torch.bool, device="cuda")
        rest[::3] = False
        assert torch.isfinite(last[:, rest]).all()
    else:
        assert not torch.isfinite(last).any()


def test_strides_of_caches_scales_and_rows():
    """Caches and scales that are parts of larger tensors, q and out with rows apart, one head of many."""
    b = make_q8([100, 45], [2, 1], 8, 2, 128, 16, HF, "int8", seed=11)
    big = lambda t: torch.zeros((t.shape[0], 3, *t.shape[1:]), dtype=t.dtype, device="cuda")  # noqa: E731
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        w = big(raw(b[n]) if n.endswith("cache") else b[n])
        w[:, 1] = raw(b[n]) if n.endswith("cache") else b[n]
        b[n] = w[:, 1].view(b[n].dtype) if n.endswith("cache") else w[:, 1]
    wide = torch.zeros((3, 8, 256), dtype=HF, device="cuda")
    wide[..., :128] = b["q"]
    b["q"] = wide[..., :128]
    out = torch.zeros((3, 16, 128), dtype=HF, device="cuda")[:, ::2]
    check_q8(attend(b, out=out), None, b)


def test_large_queries():
    """bf16 queries far outside of fp16's range, and rows with values 2^-20 of their largest."""
    b = make_q8([90, 7], [1, 1], 4, 2, 128, 16, BF, "int8", seed=12)
    b["q"] *= 2.0 ** 40
    b["q"][:, :, 3] *= 2.0 ** -20
    check_q8(attend(b, softmax_scale=2.0 ** -40 / math.sqrt(128)), None, b, scale=2.0 ** -40 / math.sqrt(128))
    b["q"] *= 2.0 ** -100
    check_q8(attend(b, softmax_scale=2.0 ** 60 / math.sqrt(128)), None, b, scale=2.0 ** 60 / math.sqrt(128))


def test_bad_pages_and_lengths_are_recorded():
    b = make_q8([40, 20], [1, 1], 4, 2, 64, 16, BF, "int8", seed=13)
    b["block_table"][0, 1] = 1 << 29
    o = attend(b)
    torch.cuda.synchronize()
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT and torch.isfinite(o).all()
    clis.clis_clear_device_error()
    b["kv_len"][1] = 1 << 20
    attend(b)
    assert clis.clis_get_device_error() & clis.PAGED_LENGTH_BIT
    clis.clis_clear_device_error()
    # more new tokens than max_q says
    b = make_q8([40], [40], 4, 2, 64, 16, BF, "int8", seed=13)
    attend(b, max_q=1)
    assert clis.clis_get_device_error() == clis.PAGED_LENGTH_BIT
    clis.clis_clear_device_error()


def test_graph_replays_other_lengths():
    b = make_q8([300, 40], [1, 1], 8, 2, 128, 16, BF, "int8", seed=14)
    o = torch.empty_like(b["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    call = lambda: clis.clis_attn_fwd_paged(b["q"], b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], b["kv_len"], 1,  # noqa: E731
                                            clis.scale_log2_for(128), out=o, workspace=ws, k_scale=b["k_scale"], v_scale=b["v_scale"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cut in (0, 7, 33):
        b["kv_len"].sub_(cut)
        want = attend(b)
        o.zero_()
        graph.replay()
        assert torch.equal(o, want)
        b["kv_len"].add_(cut)


# --------------------------------------------------------------- write, read


def turned(x, pos, inv, axis, inter):
    """x [T, H, d] rotated in 64 bits."""
    P = inv.numel()
    a = (pos.double()[:, axis.long()] * inv)[:, None]
    c, s = a.cos(), a.sin()
    x = x.double()
    y = x.clone()
    i0, i1 = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if inter else (slice(0, P), slice(P, 2 * P))
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def check_rows(got_codes, got_scale, x, code, turn):
    """Codes and scales of rows x (64 bits).  The scale: the largest magnitude, 2^-24 of it (and of the rotation's
    products, 2 * 2^-24, with sin and cos off by 2^-23) off, then one division: 2^-21 in all.  A value: half a step of its
    code, and what the scale's error makes of it."""
    top = x.abs().amax(-1)
    want = torch.where(top < 2.0 ** -100, 0.0, top / TOP[code])
    assert ((got_scale.double() - want).abs() <= 2.0 ** (-21 if turn else -23) * want).all()
    v = got_codes.float().double()
    assert (v.abs() <= TOP[code]).all()
    unit = want[..., None]
    half = 0.5 * unit if code == "int8" else torch.maximum(x.abs() * 2.0 ** -4, unit * 2.0 ** -10)
    x = torch.where(unit > 0, x, 0.0)
    assert ((v * got_scale.double()[..., None] - x).abs() <= half * (1 + 2.0 ** -16) + 2.0 ** -20 * unit * TOP[code]).all()


@pytest.mark.parametrize("T,H,Hk,d,page,pairs,axes,inter", [
    (1, 1, 1, 64, 8, 8, 1, False), (7, 16, 2, 64, 16, 32, 2, True), (65, 32, 8, 128, 16, 64, 3, True),
    (130, 6, 3, 128, 64, 24, 4, False), (33, 5, 5, 64, 32, 0, 1, False), (2049, 8, 4, 128, 8, 64, 1, False)])
@pytest.mark.parametrize("dtype,code", [(BF, "int8"), (HF, "int8"), (BF, "e4m3"), (HF, "e4m3")])
def test_write(T, H, Hk, d, page, pairs, axes, inter, dtype, code):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v = r(T, H, d), r(T, Hk, d), r(T, Hk, d)
    k[..., 5] *= 30
    k[0, 0] = 0.0
    if T > 5:
        v[3] *= 2.0 ** -14
        v[4, -1] = 0.0
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    if T > 2:
        slots[T // 2] = -1
    kc, vc = (torch.full((pages, Hk, page, d), 5, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hk, page), -1.0, device="cuda") for _ in range(2))
    inv = 10000.0 ** (-torch.arange(max(pairs, 1), dtype=torch.float64, device="cuda") / max(pairs, 1))
    axis = (torch.arange(max(pairs, 1), device="cuda") % axes).int()
    pos = torch.randint(0, 100000, (T, axes), generator=g, device="cuda", dtype=torch.int32)
    kw = {"q": q, "positions": pos, "inv_freq": inv, "axis": axis, "interleaved": inter} if pairs else {}
    got = clis.paged_append(k, v, kc.view(CODES[code]), vc.view(CODES[code]), slots, k_scale=ks, v_scale=vs, **kw)
    if pairs:
        want_q = clis.paged_append(k, v, *(torch.zeros((pages, Hk, page, d), dtype=dtype, device="cuda") for _ in range(2)), slots, **kw)
        assert torch.equal(got, want_q)  # (as beside a cache of 16-bit values)
    live = slots >= 0
    at = slots[live]
    for x, c, s, turn in ((turned(k, pos, inv, axis, inter) if pairs else k.double(), kc, ks, pairs > 0), (v.double(), vc, vs, False)):
        check_rows(c[at // page, :, at % page].view(CODES[code]), s[at // page, :, at % page], x[live], code, turn)
        rest = torch.ones((pages, page), dtype=torch.bool, device="cuda")
        rest[at // page, at % page] = False
        assert (c.transpose(1, 2)[rest] == 5).all() and (s.transpose(1, 2)[rest] == -1.0).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_write_of_non_finite_rows(code):
    k = torch.randn(6, 2, 64, device="cuda").to(BF)
    v = k.clone()
    k[1, 0, 7], k[2, 1, 63], v[3, 0, 0], v[4, 1, 30] = math.nan, math.inf, -math.inf, math.nan
    k[5] = 2.0 ** -120
    v[5] = 2.0 ** -99
    kc, vc = (torch.full((1, 2, 8, 64), 9, dtype=torch.int8, device="cuda").view(CODES[code]) for _ in range(2))
    ks, vs = (torch.zeros((1, 2, 8), device="cuda") for _ in range(2))
    clis.paged_append(k, v, kc, vc, torch.arange(6, device="cuda"), k_scale=ks, v_scale=vs)
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    k2, v2 = clis.paged_read(kc, vc, bt, cu, 6, k_scale=ks, v_scale=vs)
    for x, y in ((k, k2), (v, v2)):
        bad = ~torch.isfinite(x.float()).all(-1)
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    assert (k2[5] == 0).all() and (v2[5] == 2.0 ** -99).all()


@pytest.mark.parametrize("S,ctx,Hk,d,page,dtype,code", [
    (1, 1, 1, 64, 8, BF, "int8"), (3, 71, 4, 64, 16, HF, "e4m3"), (5, 1000, 3, 128, 32, BF, "e4m3"),
    (40, 130, 8, 128, 16, HF, "int8"), (4, 300, 2, 128, 64, BF, ""), (2, 5000, 8, 64, 8, HF, "")])
def test_read(S, ctx, Hk, d, page, dtype, code):
    lens = [ctx - (i * 37) % ctx for i in range(S)]
    lens[S // 2] = 0 if S > 2 else lens[S // 2]
    b = make_q8(lens, [0] * S, Hk, Hk, d, page, dtype, code or "int8", seed=S, layout="nhd" if S % 2 else "hnd")
    start = torch.tensor([n // 3 for n in lens], dtype=torch.int32, device="cuda")
    cnt = [n - n // 3 for n in lens]
    cu = torch.tensor([sum(cnt[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
    T = sum(cnt)
    if code:
        k, v = clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], cu, T, start=start, k_scale=b["k_scale"],
                               v_scale=b["v_scale"], dtype=dtype)
        want = [torch.cat([(c.float() * x[..., None]).to(dtype)[n // 3:] for (c, x), n in zip(w, lens)])
                for w in zip(*b["keys"])]
    else:
        kc, vc = (torch.randn(b["k_cache"].shape, device="cuda").to(dtype) for _ in range(2))
        k, v = clis.paged_read(kc, vc, b["block_table"], cu, T, start=start)
        seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(cnt, device="cuda"))
        at = start.long()[seq] + torch.arange(T, device="cuda") - cu.long()[seq]
        pg = b["block_table"].long()[seq, at // page]
        want = [kc[pg, :, at % page], vc[pg, :, at % page]]
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_read_leaves_other_rows_and_records_bad_places():
    b = make_q8([20, 9], [0, 0], 2, 2, 64, 8, BF, "int8", seed=1)
    cu = torch.tensor([0, 20, 29], dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((33, 4, 64), 3.0, dtype=BF, device="cuda")[:, ::2] for _ in range(2))
    kw = {"k_scale": b["k_scale"], "v_scale": b["v_scale"]}
    k, v = clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], cu, 33, k_out=ko, v_out=vo, **kw)
    assert k is ko and (ko[29:] == 3.0).all() and (ko[:29] != 3.0).any()
    b["block_table"][0, 1] = -5
    k2, _ = clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], cu, 29, **kw)
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
    assert (k2[8:16] == 0).all() and torch.equal(k2[:8], ko[:8]) and torch.equal(k2[16:], ko[16:29])
    clis.clis_clear_device_error()
    start = torch.tensor([0, 1 << 30], dtype=torch.int32, device="cuda")
    b["block_table"][0, 1] = 0
    k3, _ = clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], cu, 29, start=start, **kw)
    assert clis.clis_get_device_error() == clis.PAGED_LENGTH_BIT and (k3[20:] == 0).all()
    clis.clis_clear_device_error()


# ------------------------------------------------------------ sizes, streams, refusals


@pytest.mark.parametrize("n", [1, 5, 80])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_the_longest_sequence(n, code):
    """2^26 - 3 keys (one page, 1,024 times over) in one sequence, shared out over the whole GPU."""
    page, times, d = 65536, 1024, 64
    b = make_q8([page], [0], 4, 1, d, page, BF, code, seed=16, poison=False)
    q = torch.randn((n, 4, d), device="cuda").to(BF)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    at = b["block_table"][0, 0].item()
    o, lse2 = clis.attention_paged(q, b["k_cache"], b["v_cache"], torch.full((1, times), at, dtype=torch.int32, device="cuda"), i32([0, n]),
                                   i32([page * times - 3]), n, causal=True, return_lse=True, k_scale=b["k_scale"], v_scale=b["v_scale"])
    (kc, ks), (vc, vs) = b["keys"][0]
    k, v = (c[:, 0].float().double() * s.double() for c, s in ((kc, ks), (vc, vs)))
    count = torch.full((n, page), float(times), dtype=torch.float64, device="cuda")
    for i in range(n):                                  # query i is key 2^26 - 3 - n + i
        count[i, page - 3 - n + i + 1:] -= 1
    x = q.double().transpose(0, 1) @ k.T / 8.0
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m) * count
    L = p.sum(-1, keepdim=True)
    want, A = ((p @ t / L).transpose(0, 1) for t in (v, v.abs()))
    # As check_q8, for chunks also V's rounding (2^-8 of A); 32-bit sums: a run is at most 2^26 / 152 keys, 16 to a product,
    # each of which may cut off 2^-23 of the sum.
    tol = 2.0 ** -8 * (want.abs() + (2 * A if 4 * n > 64 else 0)) + (2.0 ** -11 + 6e-4) * A * 1.01
    tol = tol + want.abs() * (2.0 ** 26 / 152 / 16 * 2.0 ** -23) + 2.0 ** -32 * (vs.max() / vs.min()) * A
    assert ((o.double() - want).abs() <= tol).all()
    e = (lse2.double() - ((m + L.log())[..., 0] / math.log(2.0)).transpose(0, 1)).abs().max().item()
    assert e <= 6e-4 + 2.0 ** -22 * 32 + 2.0 ** 26 / 152 / 128 * 2.0 ** -24 / math.log(2.0), e


@pytest.mark.parametrize("d,page", [(128, 16), (64, 8), (128, 64), (64, 256)])
@pytest.mark.parametrize("dtype,code", [(BF, "int8"), (HF, "e4m3")])
def test_chunks_in_a_cache_of_many_pages(d, page, dtype, code):
    """Where the tables have fewer places than the cache pages, the chunk kernel's copies are by place: the same bits, a
    fraction of the workspace, and pages out of range are recorded as ever."""
    b = make_q8([300, 20, 0, 64], [600, 1, 0, 40], 16, 4, d, page, dtype, code, seed=page)
    assert which(b) == {"chunk"}
    check_q8(attend(b), None, b)
    wide = dict(b)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        t = b[name]
        more = torch.full((5000, *t.shape[1:]), 1, dtype=torch.int8, device="cuda").view(t.dtype) if t.dtype != torch.float32 else \
            torch.full((5000, *t.shape[1:]), math.nan, device="cuda")
        raw_t, raw_more = (raw(t), raw(more)) if t.dtype != torch.float32 else (t, more)
        wide[name] = torch.cat([raw_t, raw_more]).view(t.dtype)
    bad = b["block_table"].clone()
    bad[0, 1] = 1 << 29
    for table in (b["block_table"], bad):
        o = [attend(dict(x, block_table=table), return_lse=True) for x in (b, wide)]
        assert torch.equal(o[0][0], o[1][0]) and torch.equal(o[0][1], o[1][1])
    torch.cuda.synchronize()
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
    clis.clis_clear_device_error()
    # Both calls take the same output and the same workspace for parts of items (some 50 MB); the copies of the second have
    # S * width pages instead of the first's, 2 * 2 d + 4 bytes a row, and a table, rounded to 256 bytes (torch: 2 MB a tensor).
    used = []
    for x in (b, wide):
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        held = torch.cuda.memory_allocated()
        attend(x)
        used.append(torch.cuda.max_memory_allocated() - held)
    places, pages = b["block_table"].numel(), b["k_cache"].shape[0]
    assert used[1] - used[0] <= (places - pages) * 4 * page * (4 * d + 4) + 4 * places + (5 << 20)


def test_caches_beyond_32_bits():
    """Pages past 2^31 bytes and past 2^31 rows' worth of offsets: written, read back and attended."""
    page, Hk, d, pages = 64, 8, 128, 36000  # 2.36 GB of codes each
    kc, vc = (torch.empty((pages, Hk, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, Hk, page), device="cuda") for _ in range(2))
    T = 200
    k, v = (torch.randn((T, Hk, d), device="cuda").to(BF) for _ in range(2))
    bt = torch.tensor([[35999, 3, 35990, 35000, 0]], dtype=torch.int32, device="cuda")
    at = torch.arange(T, device="cuda")
    slots = bt[0].long()[at // page] * page + at % page
    clis.paged_append(k, v, kc, vc, slots, k_scale=ks, v_scale=vs)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k2, v2 = clis.paged_read(kc, vc, bt, i32([0, T]), T, k_scale=ks, v_scale=vs)
    for x, y in ((k, k2), (v, v2)):  # half a step of the code, and the rounding of the value read
        top = x.float().abs().amax(-1, keepdim=True)
        assert ((x.float() - y.float()).abs() <= top / 254 * 1.001 + 2.0 ** -8 * y.float().abs()).all()
    held = [(c[bt[0].long()[at // page], :, at % page], x[bt[0].long()[at // page], :, at % page]) for c, x in ((kc, ks), (vc, vs))]
    for n in (1, 3, 20):
        b = {"q": torch.randn((n, 32, d), device="cuda").to(BF), "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "block_table": bt,
             "cu_q": i32([0, n]), "kv_len": i32([T]), "keys": [held], "ctx": [T - n], "new": [n], "max_q": n}
        check_q8(attend(b), None, b)


def test_given_stream_and_workspace():
    b = make_q8([500, 90], [1, 1], 8, 2, 128, 16, BF, "int8", seed=17)
    want = attend(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = clis.clis_attn_fwd_paged(b["q"], b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], b["kv_len"], 1, clis.scale_log2_for(128),
                                 stream=side, k_scale=b["k_scale"], v_scale=b["v_scale"])
    k, v = clis.clis_paged_read(b["k_cache"], b["v_cache"], b["block_table"], torch.tensor([0, 501, 592], dtype=torch.int32, device="cuda"), 592,
                                k_scale=b["k_scale"], v_scale=b["v_scale"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want)
    (kc, ks), _ = b["keys"][0]
    assert torch.equal(k[:501], (kc.float() * ks[..., None]).to(BF))


def test_refusals_on_the_host():
    b = make_q8([50], [1], 8, 2, 64, 16, BF, "int8", seed=18)
    kw = {"k_scale": b["k_scale"], "v_scale": b["v_scale"]}
    args = [b["q"], b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], b["kv_len"], 1]

    def no(match, **change):
        a, k = list(args), dict(kw)
        for n, x in change.items():
            if n in k:
                k[n] = x
            else:
                a[int(n[1:])] = x
        with pytest.raises((ValueError, clis.ClisError), match=match):
            clis.attention_paged(*a, **k)

    no("belong together", v_scale=None)
    no("codes need k_scale", k_scale=None, v_scale=None)
    no("float32", k_scale=b["k_scale"].double())
    no("float32", k_scale=b["k_scale"][:1])
    no("int8 or float8", _1=b["k_cache"].float().to(BF), _2=b["v_cache"].float().to(BF))
    no("int8 or float8", _2=b["v_cache"].view(torch.float8_e4m3fn))
    no("MISALIGNED|multiple|aligned", _1=raw(b["k_cache"])[..., 8:].contiguous().new_zeros((b["k_cache"].shape[0], 2, 16, 72))[..., :64])
    with pytest.raises(ValueError, match="dtype"):
        clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], 1, dtype=torch.float32, **kw)
    with pytest.raises(ValueError, match="without scales"):
        clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], 1)
    with pytest.raises(ValueError, match="k_out and v_out"):
        clis.paged_read(b["k_cache"], b["v_cache"], b["block_table"], b["cu_q"], 1, k_out=torch.empty((1, 2, 64), device="cuda"), **kw)
