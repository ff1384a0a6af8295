"""Argument checks of the calls around a paged cache: everything is refused on the host, before any
CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis

FAKE = 1 << 20  # never followed: every call below is refused, or has nothing to do
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
CUDA = 5  # (what a call that would be made says on a machine without a GPU)


def rope_desc(**kw):
    d = dict(B=1, Hq=4, Hk=2, N=10, d=128, pairs=64, axes=3, interleaved=0, inverse=0, dtype=0,
             q_sb=5120, q_sh=1280, q_sn=128, k_sb=2560, k_sh=1280, k_sn=128,
             qo_sb=5120, qo_sh=1280, qo_sn=128, ko_sb=2560, ko_sh=1280, ko_sn=128, p_sb=30, p_sn=3, p_sa=1)
    d.update(kw)
    return clis.RopeDesc(**d)


def paged_desc(**kw):
    d = dict(S=3, T=10, H=4, Hkv=2, d=128, page_size=16, num_pages=50, width=8, q_st=512, q_sh=128, o_st=512, o_sh=128,
             kc_sp=4096, kc_sh=2048, kc_sn=128, vc_sp=4096, vc_sh=2048, vc_sn=128, bt_ss=8, dtype=0)
    d.update(kw)
    return clis.PagedDesc(**d)


def rope(desc, **p):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, inv=FAKE, axis=FAKE)
    a.update(p)
    return clis.load_library().clis_rope(desc, *a.values(), None)


def plan(desc, ring_size=50, **p):
    a = dict(ctx=FAKE, new=FAKE, bt=FAKE, ring=FAKE, size=ring_size, st=FAKE, so=FAKE + 64, cu=FAKE, kv=FAKE, slots=FAKE, pos=FAKE)
    a.update(p)
    return clis.load_library().clis_paged_plan(desc, *a.values(), None)


def append(desc, r, v_st=256, v_sh=128, **p):
    a = dict(q=FAKE, k=FAKE, v=FAKE, v_st=v_st, v_sh=v_sh, qo=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE, inv=FAKE, axis=FAKE)
    a.update(p)
    return clis.load_library().clis_paged_append(desc, r, *a.values(), None)


def attn(desc, max_q=4, scale=0.1, causal=1, ws=FAKE, ws_bytes=1 << 40, **p):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, cu=FAKE, kv=FAKE, o=FAKE, lse=None)
    a.update(p)
    return clis.load_library().clis_attn_fwd_paged(desc, *a.values(), max_q, scale, causal, ws, ws_bytes, None)


def test_rope_refusals():
    assert rope(None) == INVALID
    for kw, st in ((dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
                   (dict(interleaved=2), INVALID), (dict(inverse=-1), INVALID), (dict(dtype=2), INVALID),
                   (dict(d=96), UNSUPPORTED), (dict(pairs=0), INVALID), (dict(pairs=72), INVALID), (dict(pairs=12), UNSUPPORTED),
                   (dict(q_sn=132), MISALIGNED), (dict(q_sn=-128), INVALID), (dict(ko_sh=4), MISALIGNED),
                   (dict(qo_sh=0), INVALID), (dict(ko_sn=0), INVALID), (dict(qo_sn=64), INVALID),   # outputs that share memory
                   (dict(qo_sh=640), INVALID), (dict(q_sb=1 << 40), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED)):
        assert rope(rope_desc(**kw)) == st, kw
    for p in ("q", "k", "qo", "ko", "pos", "inv", "axis"):
        assert rope(rope_desc(), **{p: None}) == INVALID, p
    for p in ("q", "k", "qo", "ko"):
        assert rope(rope_desc(), **{p: FAKE + 8}) == MISALIGNED, p
    assert rope(rope_desc(), pos=FAKE + 2) == MISALIGNED and rope(rope_desc(), inv=FAKE + 4) == MISALIGNED
    # nothing to do: no pointer is looked at
    for kw in (dict(B=0), dict(N=0), dict(Hq=0, Hk=0)):
        assert rope(rope_desc(**kw), q=None, k=None, qo=None, ko=None, pos=None, inv=None, axis=None) == OK


TABLE = [(dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(width=0), INVALID), (dict(num_pages=0), INVALID),
         (dict(page_size=0), INVALID), (dict(page_size=4), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
         (dict(page_size=1 << 17), UNSUPPORTED), (dict(S=16385), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
         (dict(width=(1 << 22) + 1, bt_ss=1 << 23), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED), (dict(bt_ss=-8), INVALID)]


def test_plan_refusals():
    assert plan(None) == INVALID
    for kw, st in TABLE + [(dict(bt_ss=7), INVALID)]:
        assert plan(paged_desc(**kw)) == st, kw
    assert plan(paged_desc(), ring_size=0) == INVALID and plan(paged_desc(), ring_size=1 << 31) == UNSUPPORTED
    for p in ("ctx", "new", "bt", "ring", "st", "so", "cu", "kv", "slots", "pos"):
        assert plan(paged_desc(), **{p: None}) == INVALID, p
    assert plan(paged_desc(), so=FAKE) == INVALID  # state_out is state_in
    for p in ("ctx", "bt", "ring", "cu", "kv", "pos"):
        assert plan(paged_desc(), **{p: FAKE + 2}) == MISALIGNED, p
    assert plan(paged_desc(), slots=FAKE + 4) == MISALIGNED and plan(paged_desc(), st=FAKE + 4) == MISALIGNED


CACHE = TABLE + [(dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(H=5), INVALID), (dict(d=32), UNSUPPORTED),
                 (dict(dtype=7), INVALID), (dict(kc_sn=64), INVALID), (dict(vc_sh=4), MISALIGNED), (dict(kc_sp=-8), INVALID),
                 (dict(vc_sp=1 << 38), UNSUPPORTED)]


def test_append_refusals():
    r = rope_desc()
    assert append(None, r) == INVALID and append(paged_desc(), None) == INVALID
    for kw, st in CACHE:
        assert append(paged_desc(**kw), r) == st, kw
    for kw in (dict(kc_sh=0), dict(kc_sp=2048), dict(vc_sn=120 + 8, vc_sh=128)):  # cache rows that share memory
        assert append(paged_desc(**kw), r) == INVALID, kw
    for kw in (dict(B=2), dict(N=9), dict(Hk=1), dict(Hq=3), dict(d=64, pairs=8), dict(dtype=1), dict(inverse=1), dict(axes=0),
               dict(qo_sh=0)):
        assert append(paged_desc(), rope_desc(**kw)) == INVALID, kw
    assert append(paged_desc(), r, v_sh=4) == MISALIGNED
    for p in ("q", "k", "v", "qo", "kc", "vc", "slots", "pos", "inv", "axis"):
        assert append(paged_desc(), r, **{p: None}) == INVALID, p
    for p in ("q", "k", "v", "qo", "kc", "vc"):
        assert append(paged_desc(), r, **{p: FAKE + 8}) == MISALIGNED, p
    assert append(paged_desc(), rope_desc(pairs=0)) == INVALID  # q, and nothing to rotate it by
    assert append(paged_desc(T=0), rope_desc(N=0), q=None, k=None, v=None, kc=None, vc=None, slots=None) == OK


def test_attention_refusals():
    assert attn(None) == INVALID
    for kw, st in CACHE:
        assert attn(paged_desc(**kw)) == st, kw
    for kw, st in ((dict(q_st=64), INVALID), (dict(q_st=516), MISALIGNED), (dict(o_sh=0), INVALID), (dict(o_st=0), INVALID),
                   (dict(o_st=256), INVALID), (dict(o_sh=64), INVALID), (dict(H=258, Hkv=2, o_st=1 << 20), UNSUPPORTED),
                   (dict(S=16384, Hkv=4096, H=4096, o_st=1 << 20, width=1 << 20, bt_ss=1 << 20, kc_sp=1 << 24, vc_sp=1 << 24), UNSUPPORTED)):
        assert attn(paged_desc(**kw)) == st, kw
    assert attn(paged_desc(), max_q=0) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attn(paged_desc(), scale=scale) == INVALID
    assert attn(paged_desc(), causal=2) == INVALID
    for p in ("q", "kc", "vc", "bt", "cu", "kv", "o"):
        assert attn(paged_desc(), **{p: None}) == INVALID, p
    for p in ("q", "kc", "vc", "o"):
        assert attn(paged_desc(), **{p: FAKE + 8}) == MISALIGNED, p
    for p in ("bt", "cu", "kv", "lse"):
        assert attn(paged_desc(), **{p: FAKE + 2}) == MISALIGNED, p
    # nothing to do
    none = dict(q=None, kc=None, vc=None, bt=None, cu=None, kv=None, o=None, ws=None, ws_bytes=0)
    assert attn(paged_desc(S=0), **none) == OK and attn(paged_desc(T=0), **none) == OK
    n = ctypes.c_size_t(7)
    size = clis.load_library().clis_attn_paged_workspace_size
    assert size(paged_desc(S=0), 4, ctypes.byref(n)) == OK and n.value == 0
    assert size(None, 4, ctypes.byref(n)) == INVALID and size(paged_desc(), 4, None) == INVALID
    assert size(paged_desc(), 0, ctypes.byref(n)) == INVALID and size(paged_desc(page_size=5), 4, ctypes.byref(n)) == UNSUPPORTED


def test_status_of_bad_device_data():
    assert clis.clis_status_string(7) not in ("", "unknown status") and clis.STATUS[7] == "CLIS_ERR_DATA"


def test_python_refusals():
    """Shapes, dtypes and devices are checked before the library is called."""
    cpu = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos, inv, axis = torch.zeros(1, 4, 1, dtype=torch.int32), torch.ones(8, dtype=torch.float64), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        clis.rope(cpu, None, pos, inv, axis)
    with pytest.raises(ValueError):
        clis.paged_append(cpu[0], cpu[0], cpu, cpu, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        clis.attention_paged(cpu[0], cpu, cpu, pos[0], axis[:2], axis[:1])
    with pytest.raises(ValueError):
        clis.paged_plan(axis, axis, pos[0], axis, axis.long()[:2], 16, 4)
    with pytest.raises(ValueError):
        clis.attention(cpu, cpu, cpu, rope=clis.Rope(pos, inv, axis))


def test_the_sizes_together():
    """The limits of clis_paged_t hold together as documented: sequences x key/value heads x a table row's keys up to 2^43."""
    big = dict(S=16384, T=16384, H=8, Hkv=8, q_st=1024, o_st=1024, page_size=65536, width=1024, bt_ss=1024, num_pages=64,
               kc_sn=128, kc_sh=1 << 23, kc_sp=1 << 26, vc_sn=128, vc_sh=1 << 23, vc_sp=1 << 26)
    for d in (64, 128):
        # (no workspace: refused for that, once all sizes have been accepted)
        assert attn(paged_desc(**{**big, "d": d}), ws=None, ws_bytes=0) in (WORKSPACE, CUDA), d
        assert attn(paged_desc(**{**big, "d": d, "width": 512, "Hkv": 16, "H": 16, "q_st": 2048, "o_st": 2048}), ws=None,
                    ws_bytes=0) in (WORKSPACE, CUDA), d
        assert attn(paged_desc(**{**big, "d": d, "Hkv": 9, "H": 9, "q_st": 2048, "o_st": 2048})) == UNSUPPORTED, d


def test_angles_have_no_gradient():
    """An inv_freq that wants a gradient would silently get none: refused (unless nothing is recorded anyway)."""
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos, axis = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    inv = torch.ones(8, dtype=torch.float64, requires_grad=True)
    with pytest.raises(ValueError, match="inv_freq gets no gradient"):
        clis.rope_autograd(x, None, pos, inv, axis)
    with pytest.raises(ValueError, match="inv_freq gets no gradient"):
        clis.attention_autograd(x, x, x, rope=clis.Rope(pos, inv, axis))
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):  # (the next check: these are host tensors)
        clis.rope_autograd(x, None, pos, inv, axis)
