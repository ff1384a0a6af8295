"""Rotary positions and the write into a paged cache against 64-bit rotations."""
import math

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis
from paged_util import HALF_STEP

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def clean_error_word():
    clis.clis_clear_device_error()
    yield
    assert clis.clis_get_device_error() == 0


def table(pairs, axes, theta=10000.0):
    inv = theta ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    axis = (torch.arange(pairs) * axes // pairs).to(torch.int32)
    return inv.cuda(), axis.cuda()


def turned(x, positions, inv, axis, interleaved, sign=1.0):
    """x [..., N, d] rotated in 64 bits; positions [N, axes] or [B, 1, N, axes]."""
    P = inv.numel()
    a = positions.double()[..., axis.long()] * inv * sign
    c, s = torch.cos(a), torch.sin(a)
    x = x.double()
    y = x.clone()
    if interleaved:
        x0, x1 = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = x0 * c - x1 * s, x1 * c + x0 * s
    else:
        x0, x1 = x[..., :P], x[..., P:2 * P]
        y[..., :P], y[..., P:2 * P] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


def check(got, want, x, what=""):
    """One rounding of the result (half a step), and 32-bit arithmetic before it: the angle
    (a fraction of a turn rounded to 24 bits: 2^-24 * pi rad at most, with the double table's own
    2^-52 * |pos| below it), sin and cos (2 ulp), two products and a sum: 8 * 2^-24 of |x0| + |x1|,
    which is at most 2 max |x| of the row; fp16 results below 2^-14 round to 2^-25 at best."""
    u = HALF_STEP[got.dtype]
    big = x.double().abs().amax(-1, keepdim=True) * 2
    tol = u * want.abs() * 1.001 + 8 * 2.0 ** -24 * big + (2.0 ** -25 if got.dtype == FP else 0)
    over = ((got.double() - want).abs() / tol).max().item() if want.numel() else 0.0
    assert over <= 1.0, f"{what}: {over:.2f} times the bound"


CASES = [  # B, H, Hk, N, d, pairs, axes, interleaved, dtype, far
    (1, 1, 1, 1, 64, 8, 1, False, BF, 100),
    (1, 4, 2, 7, 128, 64, 3, True, BF, 50),
    (2, 5, 1, 33, 128, 48, 2, False, FP, 2 ** 20),
    (1, 16, 16, 129, 64, 32, 4, True, FP, 2 ** 31 - 1),
    (3, 3, 3, 257, 128, 16, 3, False, BF, 2 ** 31 - 1),
    (2, 20, 4, 1000, 128, 64, 3, True, BF, 4000),
    (1, 33, 1, 64, 64, 24, 1, False, FP, 30000),
]


@pytest.mark.parametrize("B,H,Hk,N,d,pairs,axes,interleaved,dtype,far", CASES)
def test_against_64_bits(B, H, Hk, N, d, pairs, axes, interleaved, dtype, far):
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k = (torch.randn((B, h, N, d), generator=g, device="cuda").to(dtype) for h in (H, Hk))
    pos = torch.randint(-far, far, (B, N, axes), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    inv, axis = table(pairs, axes)
    for inverse in (False, True):
        yq, yk = clis.clis_rope(q, k, pos, inv, axis, interleaved, inverse)
        for y, x in ((yq, q), (yk, k)):
            check(y, turned(x, pos[:, None], inv, axis, interleaved, -1.0 if inverse else 1.0), x)
            assert torch.equal(y[..., 2 * pairs:], x[..., 2 * pairs:])
    only, none = clis.rope(q, None, pos, inv, axis, interleaved)
    assert none is None and torch.equal(only, clis.rope(q, k, pos, inv, axis, interleaved)[0])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_strides_and_in_place(dtype):
    """[B, N, H, d] storage, broadcast heads, positions axis-major and shared, in place."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, H, Hk, N, d = 2, 6, 2, 45, 64
    q = torch.randn((B, N, H, d + 8), generator=g, device="cuda").to(dtype)[..., :d].transpose(1, 2)
    k = torch.randn((B, 1, N, d), generator=g, device="cuda").to(dtype).expand(B, Hk, N, d)
    pos = torch.randint(0, 999, (3, N), generator=g, device="cuda", dtype=torch.int32).t()
    inv, axis = table(32, 3)
    want = [turned(x, pos, inv, axis, True) for x in (q, k)]
    yq, yk = clis.rope(q, k, pos, inv, axis, True)
    check(yq, want[0], q)
    check(yk, want[1], k)
    mine = q.clone(memory_format=torch.preserve_format)
    got, _ = clis.clis_rope(mine, None, pos, inv, axis, True, q_out=mine)
    assert got is mine and torch.equal(mine, yq)
    out = torch.full((B, N, H, d), 9.0, dtype=dtype, device="cuda").transpose(1, 2)
    clis.clis_rope(q, None, pos, inv, axis, True, q_out=out)
    assert torch.equal(out, yq)


def test_bad_axis_is_recorded():
    q = torch.randn(1, 2, 5, 64, device="cuda").to(BF)
    inv, axis = table(8, 1)
    axis[3] = 4
    pos = torch.ones(1, 5, 1, dtype=torch.int32, device="cuda")
    y, _ = clis.rope(q, None, pos, inv, axis)
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
    clis.clis_clear_device_error()
    assert torch.equal(y[..., 3], q[..., 3]) and torch.equal(y[..., 11], q[..., 11])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(interleaved):
    """Against the formula (the transposed rotation) and against differences of a 64-bit loss."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, H, Hk, N, d = 2, 4, 2, 19, 64
    q0, k0 = (torch.randn((B, h, N, d), generator=g, device="cuda").to(BF) for h in (H, Hk))
    gq, gk = (torch.randn((B, h, N, d), generator=g, device="cuda").to(BF) for h in (H, Hk))
    pos = torch.randint(0, 5000, (B, N, 2), generator=g, device="cuda", dtype=torch.int32)
    inv, axis = table(24, 2)
    q, k = q0.clone().requires_grad_(), k0.clone().requires_grad_()
    y = clis.rope_autograd(q, k, pos, inv, axis, interleaved)
    dq, dk = torch.autograd.grad(y, (q, k), (gq, gk))
    check(dq, turned(gq, pos[:, None], inv, axis, interleaved, -1.0), gq)
    check(dk, turned(gk, pos[:, None], inv, axis, interleaved, -1.0), gk)
    # differences: the loss sum(g * rope(x)) is linear in x, so one difference along a direction is exact
    v = torch.randn((B, H, N, d), generator=g, device="cuda").double()
    loss = lambda x: (gq.double() * turned(x, pos[:, None], inv, axis, interleaved)).sum()
    slope = (loss(q0.double() + v) - loss(q0.double() - v)) / 2
    # dq's entries are each off by half a step at most
    room = (HALF_STEP[BF] * dq.double().abs() * v.abs()).sum() + 1e-3
    assert abs((dq.double() * v).sum() - slope) <= room
    # only one of them, an expanded gradient, the other unused
    q1 = q0.clone().requires_grad_()
    yq, _ = clis.rope_autograd(q1, k0, pos, inv, axis, interleaved)
    yq.float().sum().backward()
    check(q1.grad, turned(torch.ones_like(q0), pos[:, None], inv, axis, interleaved, -1.0), torch.ones_like(q0))
    k1 = k0.clone().requires_grad_()
    _, yk = clis.rope_autograd(q0, k1, pos, inv, axis, interleaved)
    (again,) = torch.autograd.grad(yk, k1, gk, create_graph=True)
    assert torch.equal(again, dk)
    # shared key heads: an expanded leaf collects its heads' gradients
    ks = k0[:, :1].clone().requires_grad_()
    _, yk = clis.rope_autograd(q0, ks.expand(B, Hk, N, d), pos, inv, axis, interleaved)
    (one,) = torch.autograd.grad(yk, ks, gk)
    assert torch.allclose(one.double(), dk.double().sum(1, keepdim=True), rtol=2 ** -7, atol=2 ** -6)


def test_gradients_in_odd_layouts():
    """A gradient that is a contiguous piece at an odd offset, one that is expanded, none at all; inputs
    that need none."""
    q0 = torch.randn(1, 2, 5, 64, device="cuda").to(BF)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[:, None]
    inv, axis = table(32, 1)
    big = torch.randn(2 * 5 * 64 + 1, device="cuda").to(BF)
    odd = big[1:].reshape(1, 2, 5, 64)
    q, k = q0.clone().requires_grad_(), q0.clone()
    yq, yk = clis.rope_autograd(q, k, pos, inv, axis)
    (dq,) = torch.autograd.grad(yq, q, odd)
    check(dq, turned(odd, pos, inv, axis, False, -1.0), odd)
    q, k = q0.clone().requires_grad_(), q0.clone().requires_grad_()
    yq, yk = clis.rope_autograd(q, k, pos, inv, axis)
    dq, dk = torch.autograd.grad(yk, (q, k), odd.expand(1, 2, 5, 64), allow_unused=True)
    assert dq is None
    check(dk, turned(odd, pos, inv, axis, False, -1.0), odd)
    with torch.no_grad():
        y, _ = clis.rope_autograd(q, None, pos, inv, axis)
    assert not y.requires_grad


def test_not_finite_elements_stay_in_their_pairs():
    """An inf or NaN reaches its own pair and nothing else, the elements that pass through least of all."""
    inv, axis = table(16, 1)
    pos = torch.arange(1, 4, dtype=torch.int32, device="cuda")[:, None]
    for inter in (False, True):
        x = torch.ones(1, 1, 3, 64, device="cuda").to(BF)
        x[..., 40] = float("inf")
        x[..., 3] = float("nan")
        y, _ = clis.rope(x, None, pos, inv, axis, inter)
        mate = 2 if inter else 19
        bad = {3, mate, 40}
        rest = [c for c in range(64) if c not in bad]
        assert torch.isfinite(y[..., rest].float()).all() and torch.isnan(y[..., [3, mate]].float()).all()
        assert torch.isinf(y[..., 40].float()).all()


def test_training_step_captured():
    """Forward and backward of the rotation in one captured graph (no eager graph of the leaf alive: torch
    would tie the leaf's gradient to that graph's stream, which is not being captured)."""
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((1, 4, 33, 64), generator=g, device="cuda").to(BF).requires_grad_()
    gq = torch.randn((1, 4, 33, 64), generator=g, device="cuda").to(BF)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")[:, None]
    inv, axis = table(32, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            y, _ = clis.rope_autograd(q, None, pos, inv, axis)
            torch.autograd.grad(y, q, gq)
            del y
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = clis.rope_autograd(q, None, pos, inv, axis)
        (dq,) = torch.autograd.grad(y, q, gq)
    pos.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    check(y.detach(), turned(q.detach(), pos, inv, axis, False), q.detach())
    check(dq, turned(gq, pos, inv, axis, False, -1.0), gq)


def test_attention_with_rope():
    """attention and attention_autograd rotate q and k first."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((1, 4, 300, 128), generator=g, device="cuda").to(BF) for _ in range(3))
    pos = torch.stack(torch.meshgrid(torch.arange(3), torch.arange(10), torch.arange(10), indexing="ij"), -1)
    pos = pos.reshape(300, 3).to(torch.int32).cuda()
    r = clis.Rope(pos, *table(64, 3), True)
    q2, k2 = clis.rope(q, k, *r)
    assert torch.equal(clis.attention(q, k, v, rope=r), clis.attention(q2, k2, v))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    clis.attention_autograd(*leaves, causal=True, rope=r).float().square().sum().backward()
    plain = [t.clone().requires_grad_() for t in (q2, k2, v)]
    clis.attention_autograd(*plain, causal=True).float().square().sum().backward()
    want_q, want_k = clis.clis_rope(plain[0].grad, plain[1].grad, *r, inverse=True)
    assert torch.equal(leaves[0].grad, want_q) and torch.equal(leaves[1].grad, want_k)
    assert torch.equal(leaves[2].grad, plain[2].grad)


def test_graph_and_stream():
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k = (torch.randn((1, 4, 50, 64), generator=g, device="cuda").to(FP) for _ in range(2))
    pos = torch.randint(0, 99, (50, 1), generator=g, device="cuda", dtype=torch.int32)
    inv, axis = table(32, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, yk = clis.rope(q, k, pos, inv, axis)
    pos.add_(7)
    graph.replay()
    torch.cuda.synchronize()
    wq, wk = clis.rope(q, k, pos, inv, axis)
    assert torch.equal(yq, wq) and torch.equal(yk, wk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sq, _ = clis.clis_rope(q, k, pos, inv, axis, stream=side)
    side.synchronize()
    assert torch.equal(sq, wq)


# ------------------------------------------------------------------- append


@pytest.mark.parametrize("T,H,Hk,d,page,pairs,axes,interleaved,dtype", [
    (1, 4, 1, 128, 16, 64, 1, False, BF),
    (37, 8, 2, 64, 8, 16, 3, True, FP),
    (500, 5, 5, 128, 256, 40, 2, False, FP),
    (64, 32, 8, 128, 64, 64, 3, True, BF),
])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_append(T, H, Hk, d, page, pairs, axes, interleaved, dtype, layout):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(dtype) for h in (H, Hk, Hk))
    pages = -(-T // page) + 2
    shape = (pages, Hk, page, d) if layout == "hnd" else (pages, page, Hk, d)
    kc, vc = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if layout == "nhd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kc0, vc0 = kc.clone(), vc.clone()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    slots[T // 2] = -1
    if T > 5:
        slots[1] = -(2 ** 62)
    pos = torch.randint(-9, 10 ** 6, (T, axes), generator=g, device="cuda", dtype=torch.int32)
    inv, axis = table(pairs, axes)
    y = clis.paged_append(k, v, kc, vc, slots, q=q, positions=pos, inv_freq=inv, axis=axis, interleaved=interleaved)
    check(y, turned(q, pos[:, None], inv, axis, interleaved), q)
    keep = slots >= 0
    at = slots[keep]
    flat = lambda c: c.transpose(1, 2).reshape(pages * page, Hk, d)
    check(flat(kc)[at], turned(k, pos[:, None], inv, axis, interleaved)[keep], k[keep])
    assert torch.equal(flat(vc)[at], v[keep])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(flat(kc)[rest], flat(kc0)[rest]) and torch.equal(flat(vc)[rest], flat(vc0)[rest])
    # the same rotation as clis.rope, bit for bit
    yq, yk = clis.rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None], pos, inv, axis, interleaved)
    assert torch.equal(y, yq[0].transpose(0, 1)) and torch.equal(flat(kc)[at], yk[0].transpose(0, 1)[keep])
    # without rotation, and q in place
    assert clis.paged_append(k, v, kc, vc, slots) is None
    assert torch.equal(flat(kc)[at], k[keep])
    q2 = q.clone()
    assert clis.paged_append(k, v, kc, vc, slots, q=q2, positions=pos, inv_freq=inv, axis=axis,
                             interleaved=interleaved, q_out=q2) is q2
    assert torch.equal(q2, y)


def test_append_slot_out_of_range_is_recorded():
    k = torch.randn(3, 2, 64, device="cuda").to(BF)
    kc = torch.zeros(2, 2, 8, 64, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    clis.paged_append(k, k, kc, vc, torch.tensor([16, 3, 2 ** 61], device="cuda"))
    assert clis.clis_get_device_error() == clis.PAGED_INDEX_BIT
    clis.clis_clear_device_error()
    assert torch.equal(kc[0, :, 3], k[1]) and kc.abs().sum(-1).gt(0).sum() == 2


def test_append_past_32_bits():
    pages, page = 70000, 256
    kc = torch.empty((pages, 2, page, 128), dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    k, v = (torch.randn(4, 2, 128, device="cuda").to(BF) for _ in range(2))
    slots = torch.tensor([pages * page - 1, 0, (pages - 2) * page + 5, 40000 * page], device="cuda")
    clis.paged_append(k, v, kc, vc, slots)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], k[t]) and torch.equal(vc[s // page, :, s % page], v[t])


def busy(n):
    """Some milliseconds of work on the current stream."""
    a = torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    for _ in range(n):
        torch.mm(a, a, out=b)


@pytest.mark.parametrize("op", ["rope", "append", "attention", "plan"])
def test_given_stream_leaves_memory_that_is_still_read(op):
    """A tensor is dropped while a copy of it waits on the current stream: its memory is
    free for that stream's next calls, but not for a call on another stream."""
    g = torch.Generator(device="cuda").manual_seed(31)
    T, H, d = 5003, 8, 128
    side = torch.cuda.Stream()
    if op == "plan":
        lens = [torch.tensor([n], dtype=torch.int32, device="cuda") for n in (0, 300_007)]
        bt = torch.full((1, 1200), -1, dtype=torch.int32, device="cuda")
        ring = torch.arange(1200, dtype=torch.int32, device="cuda")
        state = torch.tensor([0, 1200], dtype=torch.int64, device="cuda")
        like = torch.empty(300_007, dtype=torch.int64, device="cuda")
        call = lambda s: clis.paged_plan(*lens, bt, ring, state, 256, 300_007, stream=s).slots
    else:
        like = torch.randn((T, H, d), generator=g, device="cuda").to(BF)
        q = like.clone()
        kc, vc = (torch.randn((20, 2, 256, d), generator=g, device="cuda").to(BF) for _ in range(2))
        pos = torch.arange(T, device="cuda", dtype=torch.int32)[:, None]
        inv, axis = table(64, 1)
        cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [T]))
        bt = torch.arange(20, dtype=torch.int32, device="cuda")[None]
        slots = torch.arange(T, device="cuda")
        k, v = (torch.randn((T, 2, d), generator=g, device="cuda").to(BF) for _ in range(2))
        if op == "rope":
            call = lambda s: clis.clis_rope(q[None].transpose(1, 2), None, pos, inv, axis, stream=s)[0]
        elif op == "append":
            call = lambda s: clis.paged_append(k, v, kc, vc, slots, q=q, positions=pos, inv_freq=inv, axis=axis, stream=s)
        else:
            call = lambda s: clis.clis_attn_fwd_paged(q, kc, vc, bt, cu, kv, T, 0.1, stream=s)
    busy(1)
    want = call(None).clone()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    for _ in range(3):
        x = torch.full_like(like, 7)
        y = torch.empty_like(x)
        torch.cuda.synchronize()
        busy(40)
        y.copy_(x)
        del x
        got = call(side)
        torch.cuda.synchronize()
        assert (y == 7).all(), "the dropped tensor's memory was written before it was read"
        assert torch.equal(got, want)
        del got, y


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_in_fp16(interleaved):
    """Against the formula, with the positions of a long text, all pairs and part of them."""
    g = torch.Generator(device="cuda").manual_seed(13)
    B, H, Hk, N, d = 1, 3, 1, 77, 128
    for pairs in (64, 24):
        q, k = (torch.randn((B, h, N, d), generator=g, device="cuda").to(FP).requires_grad_() for h in (H, Hk))
        gq, gk = (torch.randn((B, h, N, d), generator=g, device="cuda").to(FP) for h in (H, Hk))
        pos = torch.randint(0, 10 ** 6, (N, 1), generator=g, device="cuda", dtype=torch.int32)
        inv, axis = table(pairs, 1)
        dq, dk = torch.autograd.grad(clis.rope_autograd(q, k, pos, inv, axis, interleaved), (q, k), (gq, gk))
        check(dq, turned(gq, pos, inv, axis, interleaved, -1.0), gq)
        check(dk, turned(gk, pos, inv, axis, interleaved, -1.0), gk)
        assert dq.dtype == FP and torch.equal(dq[..., 2 * pairs:], gq[..., 2 * pairs:])
