"""Argument checks of the calls around a cache in 8 bits and of beam search: everything is refused on the host,
before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

from certified_fixed_stabilizer_gb300 import clis
from test_paged_abi import CACHE, CUDA, FAKE, INVALID, MISALIGNED, OK, TABLE, UNSUPPORTED, WORKSPACE, paged_desc, rope_desc


def quant(**kw):
    d = dict(code=0, ks_sp=32, ks_sh=16, ks_sn=1, vs_sp=32, vs_sh=16, vs_sn=1)
    d.update(kw)
    return clis.QuantDesc(**d)


def append(desc, z, r, v_st=256, v_sh=128, **p):
    a = dict(q=FAKE, k=FAKE, v=FAKE, v_st=v_st, v_sh=v_sh, qo=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, pos=FAKE, inv=FAKE,
             axis=FAKE)
    a.update(p)
    return clis.load_library().clis_paged_append_q8(desc, z, r, *a.values(), None)


def read(desc, z, k_st=256, k_sh=128, v_st=256, v_sh=128, **p):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cu=FAKE, start=FAKE, ko=FAKE, k_st=k_st, k_sh=k_sh, vo=FAKE, v_st=v_st, v_sh=v_sh)
    a.update(p)
    return clis.load_library().clis_paged_read(desc, z, *a.values(), None)


def attn(desc, z, max_q=4, scale=0.1, causal=1, ws=FAKE, ws_bytes=1 << 50, **p):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cu=FAKE, kv=FAKE, o=FAKE, lse=None)
    a.update(p)
    return clis.load_library().clis_attn_fwd_paged_q8(desc, z, *a.values(), max_q, scale, causal, ws, ws_bytes, None)


QUANT = [(dict(code=2), INVALID), (dict(code=-1), INVALID), (dict(ks_sp=-1), INVALID), (dict(vs_sn=-1), INVALID),
         (dict(vs_sp=1 << 38), UNSUPPORTED)]
CODES = [(dict(kc_sn=136, kc_sh=4096, kc_sp=8192), MISALIGNED), (dict(vc_sp=4104), MISALIGNED),   # multiples of 16, not of 8
         (dict(kc_sh=0), INVALID), (dict(vc_sp=2048), INVALID)]                                  # rows that share memory


def test_append_refusals():
    r = rope_desc()
    assert append(None, quant(), r) == INVALID and append(paged_desc(), None, r) == INVALID and append(paged_desc(), quant(), None) == INVALID
    for kw, st in CACHE + CODES:
        assert append(paged_desc(**kw), quant(), r) == st, kw
    for kw, st in QUANT + [(dict(ks_sn=0), INVALID), (dict(vs_sh=8), INVALID), (dict(ks_sp=0), INVALID)]:  # scales that share memory
        assert append(paged_desc(), quant(**kw), r) == st, kw
    for p in ("q", "k", "v", "qo", "kc", "vc", "ks", "vs", "slots", "pos", "inv", "axis"):
        assert append(paged_desc(), quant(), r, **{p: None}) == INVALID, p
    for p in ("kc", "vc"):
        assert append(paged_desc(), quant(), r, **{p: FAKE + 8}) == MISALIGNED, p
    for p in ("ks", "vs"):
        assert append(paged_desc(), quant(), r, **{p: FAKE + 2}) == MISALIGNED, p
    assert append(paged_desc(T=0), quant(), rope_desc(N=0), q=None, k=None, v=None, kc=None, vc=None, ks=None, vs=None, slots=None) == OK


def test_read_refusals():
    assert read(None, quant()) == INVALID
    for kw, st in TABLE + CODES + [(dict(Hkv=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(kc_sn=64), INVALID),
                                   (dict(T=(1 << 27) + 1), UNSUPPORTED)]:
        assert read(paged_desc(**kw), quant()) == st, kw
    for kw, st in QUANT:
        assert read(paged_desc(), quant(**kw)) == st, kw
    for kw, st in ((dict(k_st=260), MISALIGNED), (dict(v_sh=4), MISALIGNED), (dict(k_sh=-8), INVALID), (dict(k_st=128), INVALID),
                   (dict(v_sh=64), INVALID), (dict(v_st=0), INVALID), (dict(k_st=1 << 38), UNSUPPORTED)):
        assert read(paged_desc(), quant(), **kw) == st, kw
    for p in ("kc", "vc", "ks", "vs", "bt", "cu", "ko", "vo"):
        assert read(paged_desc(), quant(), **{p: None}) == INVALID, p
    for p in ("kc", "vc", "ko", "vo"):
        assert read(paged_desc(), quant(), **{p: FAKE + 8}) == MISALIGNED, p
    for p in ("ks", "vs", "bt", "cu", "start"):
        assert read(paged_desc(), quant(), **{p: FAKE + 2}) == MISALIGNED, p
    none = dict(kc=None, vc=None, ks=None, vs=None, bt=None, cu=None, start=None, ko=None, vo=None)
    assert read(paged_desc(S=0), quant(), **none) == OK and read(paged_desc(T=0), None, **none) == OK
    assert read(paged_desc(kc_sn=136, kc_sh=2176, kc_sp=4352), None, ks=None, vs=None, ko=None) == INVALID  # (8 is enough for 16-bit values)


def test_attention_refusals():
    assert attn(None, quant()) == INVALID and attn(paged_desc(), None) == INVALID
    for kw, st in CACHE + CODES:
        assert attn(paged_desc(**kw), quant()) == st, kw
    for kw, st in QUANT:
        assert attn(paged_desc(), quant(**kw)) == st, kw
    for kw, st in ((dict(q_st=64), INVALID), (dict(q_st=516), MISALIGNED), (dict(o_sh=0), INVALID), (dict(H=258, Hkv=2, o_st=1 << 20), UNSUPPORTED)):
        assert attn(paged_desc(**kw), quant()) == st, kw
    # (a 16-bit copy of 2^40 values would not fit anything)
    assert attn(paged_desc(num_pages=(1 << 31) - 1025, page_size=64, kc_sh=8192, vc_sh=8192, kc_sp=16384, vc_sp=16384), quant()) == UNSUPPORTED
    for kw in (dict(max_q=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2)):
        assert attn(paged_desc(), quant(), **kw) == INVALID, kw
    for p in ("q", "kc", "vc", "ks", "vs", "bt", "cu", "kv", "o"):
        assert attn(paged_desc(), quant(), **{p: None}) == INVALID, p
    for p in ("q", "kc", "vc", "o"):
        assert attn(paged_desc(), quant(), **{p: FAKE + 8}) == MISALIGNED, p
    for p in ("ks", "vs", "bt", "cu", "kv", "lse"):
        assert attn(paged_desc(), quant(), **{p: FAKE + 2}) == MISALIGNED, p
    assert attn(paged_desc(), quant(), ws=None, ws_bytes=0) in (WORKSPACE, CUDA)
    none = dict(q=None, kc=None, vc=None, ks=None, vs=None, bt=None, cu=None, kv=None, o=None, ws=None, ws_bytes=0)
    assert attn(paged_desc(S=0), quant(), **none) == OK and attn(paged_desc(T=0), quant(), **none) == OK
    n = ctypes.c_size_t(7)
    size = clis.load_library().clis_attn_paged_q8_workspace_size
    assert size(paged_desc(S=0), quant(), 4, ctypes.byref(n)) == OK and n.value == 0
    assert size(None, quant(), 4, ctypes.byref(n)) == INVALID and size(paged_desc(), None, 4, ctypes.byref(n)) == INVALID
    assert size(paged_desc(), quant(), 4, None) == INVALID and size(paged_desc(), quant(), 0, ctypes.byref(n)) == INVALID


def test_plan_of_beams_refusals():
    def plan(desc, beams):
        return clis.load_library().clis_paged_plan_beams(desc, beams, *[FAKE + 64 * i for i in range(4)], 50, *[FAKE + 64 * i for i in range(4, 10)], None)

    for beams, S, st in ((0, 3, INVALID), (-1, 3, INVALID), (2, 3, INVALID), (4, 6, INVALID), (7, 6, INVALID), (16385, 0, UNSUPPORTED)):
        assert plan(paged_desc(S=S), beams) == st, beams
    assert plan(None, 1) == INVALID


def beam(desc, ws=FAKE, ws_bytes=1 << 50, **p):
    a = dict(logits=FAKE, scores=FAKE, out=FAKE, parent=FAKE, token=FAKE)
    a.update(p)
    return clis.load_library().clis_beam_select(desc, *a.values(), ws, ws_bytes, None)


def beam_desc(**kw):
    d = dict(R=2, W=4, V=1000, K=8, dtype=0, l_sr=4000, l_sw=1000)
    d.update(kw)
    return clis.BeamDesc(**d)


def test_beam_refusals():
    assert beam(None) == INVALID
    for kw, st in ((dict(R=-1), INVALID), (dict(W=0), INVALID), (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(dtype=3), INVALID),
                   (dict(dtype=-1), INVALID), (dict(l_sr=-1), INVALID), (dict(l_sw=-1), INVALID), (dict(W=65), UNSUPPORTED),
                   (dict(K=65), UNSUPPORTED), (dict(R=65536), UNSUPPORTED), (dict(R=16384), UNSUPPORTED), (dict(V=1 << 31), UNSUPPORTED),
                   (dict(V=1 << 29), UNSUPPORTED), (dict(l_sw=1 << 38), UNSUPPORTED)):
        assert beam(beam_desc(**kw)) == st, kw
    for p in ("logits", "scores", "out", "parent", "token"):
        assert beam(beam_desc(), **{p: None}) == INVALID, p
    assert beam(beam_desc(), logits=FAKE + 1) == MISALIGNED and beam(beam_desc(dtype=2), logits=FAKE + 2) == MISALIGNED
    for p in ("scores", "out", "parent", "token"):
        assert beam(beam_desc(), **{p: FAKE + 2}) == MISALIGNED, p
    assert beam(beam_desc(), ws=None, ws_bytes=0) in (WORKSPACE, CUDA)
    assert beam(beam_desc(R=0), ws=None, ws_bytes=0, logits=None, scores=None, out=None, parent=None, token=None) == OK
    n = ctypes.c_size_t(7)
    size = clis.load_library().clis_beam_workspace_size
    assert size(beam_desc(R=0), ctypes.byref(n)) == OK and n.value == 0
    assert size(None, ctypes.byref(n)) == INVALID and size(beam_desc(), None) == INVALID and size(beam_desc(K=0), ctypes.byref(n)) == INVALID


def pages(**kw):
    d = dict(base=FAKE, layers=2, heads=3, row_bytes=256, sl=1 << 20, sp=12288, sh=4096, sn=256)
    d.update(kw)
    return (clis.PagesDesc * 1)(clis.PagesDesc(**d))


def reorder_desc(**kw):
    d = dict(groups=2, beams=3, width=8, page_size=16, num_pages=50, bt_ss=8, bo_ss=8)
    d.update(kw)
    return clis.ReorderDesc(**d)


def reorder(desc, ring_size=50, tensors=None, n=0, ws=FAKE, ws_bytes=1 << 50, **p):
    a = dict(lens=FAKE, parent=FAKE, bt=FAKE, out=FAKE + 4096, ring=FAKE, size=ring_size, st=FAKE, so=FAKE + 64, lo=FAKE + 128, done=FAKE)
    a.update(p)
    return clis.load_library().clis_paged_reorder(desc, *a.values(), tensors, n, ws, ws_bytes, None)


def test_reorder_refusals():
    assert reorder(None) == INVALID
    for kw, st in ((dict(groups=-1), INVALID), (dict(beams=0), INVALID), (dict(width=0), INVALID), (dict(num_pages=0), INVALID),
                   (dict(page_size=0), INVALID), (dict(page_size=12), UNSUPPORTED), (dict(beams=65), UNSUPPORTED),
                   (dict(groups=8192), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED), (dict(width=1 << 23, bt_ss=1 << 23, bo_ss=1 << 23), UNSUPPORTED),
                   (dict(bo_ss=7), INVALID), (dict(bt_ss=-1), INVALID)):
        assert reorder(reorder_desc(**kw)) == st, kw
    assert reorder(reorder_desc(), ring_size=0) == INVALID and reorder(reorder_desc(), ring_size=1 << 31) == UNSUPPORTED
    for p in ("lens", "parent", "bt", "out", "ring", "st", "so", "lo", "done"):
        assert reorder(reorder_desc(), **{p: None}) == INVALID, p
    for p in ("lens", "parent", "bt", "out", "ring", "lo", "done"):
        assert reorder(reorder_desc(), **{p: FAKE + 2}) == MISALIGNED, p
    assert reorder(reorder_desc(), so=FAKE) == INVALID and reorder(reorder_desc(), st=FAKE + 4) == MISALIGNED
    assert reorder(reorder_desc(bt_ss=16), out=FAKE) == INVALID  # in place with another stride
    for p in ("lens", "parent"):  # inputs of all blocks
        assert reorder(reorder_desc(), **{p: FAKE + 64}, lo=FAKE + 64) == INVALID
    assert reorder(reorder_desc(), n=-1) == INVALID and reorder(reorder_desc(), n=1) == INVALID
    assert reorder(reorder_desc(), tensors=pages(), n=9) == UNSUPPORTED
    for kw, st in ((dict(base=None), INVALID), (dict(layers=-1), INVALID), (dict(heads=-1), INVALID), (dict(row_bytes=0), INVALID),
                   (dict(row_bytes=2), INVALID), (dict(sn=252), INVALID), (dict(sp=-4), INVALID), (dict(sl=1 << 40), UNSUPPORTED),
                   (dict(row_bytes=254), MISALIGNED), (dict(sh=4098), MISALIGNED), (dict(base=FAKE + 2), MISALIGNED),
                   (dict(row_bytes=65540, sn=65540), UNSUPPORTED), (dict(heads=65537), UNSUPPORTED)):
        assert reorder(reorder_desc(), tensors=pages(**kw), n=1) == st, kw
    assert reorder(reorder_desc(), tensors=pages(), n=1, ws=None, ws_bytes=0) == WORKSPACE
    assert reorder(reorder_desc(), ws=FAKE + 16) == MISALIGNED
    n = ctypes.c_size_t(7)
    size = clis.load_library().clis_paged_reorder_workspace_size
    assert size(reorder_desc(groups=0), ctypes.byref(n)) == OK and n.value == 0
    assert size(reorder_desc(), ctypes.byref(n)) == OK and n.value >= 2 * 8 + 6 * 16 + 6 * 8 * 4
    assert size(None, ctypes.byref(n)) == INVALID and size(reorder_desc(), None) == INVALID


def test_python_refusals():
    """Shapes, dtypes and devices are checked before the library is called."""
    cpu, codes = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 4, 64, dtype=torch.int8)
    i32, f32 = torch.zeros(4, dtype=torch.int32), torch.zeros(1, 2, 4)
    with pytest.raises(ValueError):
        clis.paged_append(cpu[0], cpu[0], codes, codes, i32.long()[:2], k_scale=f32, v_scale=f32)
    with pytest.raises(ValueError):
        clis.attention_paged(cpu[0], codes, codes, i32[None], i32[:2], i32[:1], k_scale=f32, v_scale=f32)
    with pytest.raises(ValueError):
        clis.paged_read(codes, codes, i32[None], i32[:2], 3, k_scale=f32, v_scale=f32)
    with pytest.raises(ValueError, match="dtype must be"):
        clis.paged_read(codes, codes, i32[None], i32[:2], 3, k_scale=f32, v_scale=f32, dtype=torch.float32)
    with pytest.raises(ValueError):
        clis.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        clis.paged_reorder(i32, i32[None], i32[:, None], i32, i32.long()[:2], page_size=16)
    with pytest.raises(ValueError, match="page_size is needed"):
        clis.paged_reorder(i32, i32[None], i32[:, None], i32, i32.long()[:2])
