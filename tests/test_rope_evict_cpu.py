"""Rotary tables and argument checks of the rotary, insert, weighted
attention, selection and compaction calls: host code only, nothing is
enqueued."""

import ctypes
from decimal import Decimal, getcontext

import numpy as np
import pytest

ARG, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def tq():
    from turboquant_bit_kv_gb300 import build_lib, tq as mod
    build_lib.build()
    mod.lib()
    return mod


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (96, 1e6), (64, 500000.0), (32, 1.5)])
def test_turns_are_the_frequencies(tq, rot, base):
    getcontext().prec = 60
    r = tq.tq_rope_load(rot, base)
    assert (r.head_dim, r.rot_dim, r.axes) == (128, rot, 1)
    for i in range(rot // 2):
        f = Decimal(float(np.power(base, -2.0 * i / rot)))
        want = f / (2 * PI) * 2**64
        # the frequency is a double: two pow() may differ by an ulp (2^-52 of f); the product adds below a unit
        assert abs(Decimal(r.turn[i]) - want) <= want * Decimal(2)**-52 + 2
    for i in range(rot // 2, 64):
        assert r.turn[i] == 0


def test_set_freqs_is_exact_and_modulo_one_turn(tq):
    getcontext().prec = 60
    r = tq.tq_rope_load(32)
    freqs = [0.0, 1.0, -1.0, 1000.0, -7.25, 1e-12, 2.0**-70, 6.283185307179586] + [0.1 * i for i in range(8)]
    tq.tq_rope_set_freqs(r, freqs)
    for i, f in enumerate(freqs):
        want = Decimal(f) / (2 * PI) * 2**64
        diff = (Decimal(r.turn[i]) - want) % 2**64
        assert min(diff, 2**64 - diff) <= 2, (f, r.turn[i])
    for bad in (float("nan"), float("inf"), 2000.0):
        with pytest.raises(tq.TQError):
            tq.tq_rope_set_freqs(r, [bad] * 16)


def test_axes_of_the_pairs(tq):
    assert list(tq.tq_rope_load(128, sections=[16, 24, 24]).axis) == [0] * 16 + [1] * 24 + [2] * 24
    assert list(tq.tq_rope_load(32, sections=[0, 16]).axis)[:16] == [1] * 16
    a = list(tq.tq_rope_load(128, sections=[24, 20, 20], interleaved=True).axis)
    assert a == [i % 3 if i < 60 else 0 for i in range(64)]
    assert [a.count(x) for x in (0, 1, 2)] == [24, 20, 20]
    assert list(tq.tq_rope_load(128, sections=[64], interleaved=True).axis) == [0] * 64


def test_rope_refusals(tq):
    for kw in (dict(rot_dim=48), dict(rot_dim=0), dict(rot_dim=160), dict(style=2), dict(head_dim=64),
               dict(sections=[16, 16, 16, 16]), dict(sections=[])):
        with pytest.raises(tq.TQError) as e:
            tq.tq_rope_load(**kw)
        assert e.value.status == UNSUPPORTED, kw
    for kw in (dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(sections=[63]),
               dict(sections=[-1, 65]), dict(sections=[10, 30, 24], interleaved=True)):
        with pytest.raises(tq.TQError) as e:
            tq.tq_rope_load(**kw)
        assert e.value.status == ARG, kw


P = ctypes.c_void_p
A, B, C, D_ = P(1 << 20), P(2 << 20), P(3 << 20), P(4 << 20)     # aligned addresses that are never read
ODD = P((1 << 20) + 2)


def _apply(tq, **kw):
    a = dict(x=A, dtype=tq.TQ_BF16, n=4, heads=2, xt=256, xh=128, pos=B, pa=4, rope=tq.tq_rope_load(), out=C, ot=256,
             oh=128)
    a.update(kw)
    r = a["rope"]
    return tq.lib().tq_rope_apply(a["x"], a["dtype"], a["n"], a["heads"], a["xt"], a["xh"], a["pos"], a["pa"],
                                  None if r is None else ctypes.byref(r), a["out"], a["ot"], a["oh"], None)


def _bent(tq, **kw):
    r = tq.tq_rope_load()
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_apply_refusals(tq):
    assert _apply(tq, n=0) == 0
    for kw in (dict(x=None), dict(pos=None), dict(out=None), dict(rope=None), dict(n=-1), dict(heads=0), dict(xt=-256),
               dict(oh=64), dict(ot=64), dict(pa=-1)):
        assert _apply(tq, **kw) == ARG, kw
    for kw in (dict(x=ODD), dict(out=ODD), dict(xt=257), dict(oh=132), dict(pos=P((1 << 20) + 4))):
        assert _apply(tq, **kw) == ALIGN, kw
    bad = tq.tq_rope_load()
    bad.axis[3] = 1
    for kw in (dict(dtype=7), dict(rope=_bent(tq, rot_dim=40)), dict(rope=_bent(tq, axes=4)), dict(rope=bad),
               dict(rope=_bent(tq, style=5)), dict(rope=_bent(tq, head_dim=64))):
        assert _apply(tq, **kw) == UNSUPPORTED, kw


def _insert(tq, **kw):
    a = dict(k=A, kt=256, kh=128, v=B, vt=256, vh=128, dtype=tq.TQ_BF16, n=4, heads=2, pos=C, pa=4,
             rope=tq.tq_rope_load(), kcb=tq.tq_codebook_load(128, 4), vcb=tq.tq_codebook_load(128, 2), kb=C, vb=D_,
             nb=64, dst=A, hs=8)
    a.update(kw)
    ref = {n: None if a[n] is None else ctypes.byref(a[n]) for n in ("rope", "kcb", "vcb")}
    return tq.lib().tq_insert_kv(a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["dtype"], a["n"], a["heads"],
                                 a["pos"], a["pa"], ref["rope"], ref["kcb"], ref["vcb"], tq.tq_signs(), a["kb"],
                                 a["vb"], a["nb"], a["dst"], a["hs"], None)


def test_insert_refusals(tq):
    assert _insert(tq, n=0) == 0
    assert _insert(tq, k=None, kb=None, v=None, vb=None) == 0
    for kw in (dict(n=-1), dict(heads=0), dict(nb=-1), dict(hs=-1), dict(k=None), dict(vb=None), dict(kcb=None),
               dict(vcb=None), dict(pos=None), dict(dst=None), dict(kt=-256), dict(vh=-128), dict(pa=-4)):
        assert _insert(tq, **kw) == ARG, kw
    for kw in (dict(k=ODD), dict(v=ODD), dict(kt=260), dict(vh=4), dict(kb=P((1 << 20) + 1)), dict(dst=ODD),
               dict(pos=ODD)):
        assert _insert(tq, **kw) == ALIGN, kw
    off = tq.tq_codebook_load(128, 3)
    off.boundaries[2] = off.boundaries[3]           # two boundaries in one cell of the quantiser
    edge = tq.tq_codebook_load(128, 2)
    edge.boundaries[2] = 4.5 / 63                   # on a cell's edge
    nan = tq.tq_codebook_load(128, 2)
    nan.boundaries[0] = float("nan")
    for kw in (dict(dtype=3), dict(kcb=tq.tq_codebook_load(128, 8)), dict(vcb=tq.tq_codebook_load(64, 4)),
               dict(kcb=off), dict(vcb=edge), dict(vcb=nan), dict(rope=_bent(tq, rot_dim=16))):
        assert _insert(tq, **kw) == UNSUPPORTED, kw


def _attend(tq, **kw):
    a = dict(q=A, qd=tq.TQ_BF16, k=B, kcb=tq.tq_codebook_load(128, 4), v=C, vcb=tq.tq_codebook_load(128, 2), table=None,
             mp=0, page=0, lens=None, B=2, Hq=8, Hkv=2, T_cap=64, T=50, scale=0.1, w=D_, ws=50, decay=1.0, out=A,
             od=tq.TQ_F32, work=B, bytes=None)
    a.update(kw)
    n = tq.tq_attn_weights_workspace_bytes(a["B"], a["Hq"], a["Hkv"], a["T"]) if a["bytes"] is None else a["bytes"]
    ref = {m: None if a[m] is None else ctypes.byref(a[m]) for m in ("kcb", "vcb")}
    return tq.lib().tq_attn_decode_weights(a["q"], a["qd"], a["k"], ref["kcb"], a["v"], ref["vcb"], a["table"],
                                           a["mp"], a["page"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["T_cap"], a["T"],
                                           a["scale"], tq.tq_signs(), a["w"], a["ws"], a["decay"], a["out"], a["od"],
                                           a["work"], n, None)


def test_attend_refusals(tq):
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(w=None), dict(out=None), dict(work=None), dict(kcb=None),
               dict(vcb=None), dict(B=0), dict(Hq=7), dict(Hkv=0), dict(T=0), dict(T=65, ws=65), dict(T_cap=52),
               dict(ws=49), dict(scale=float("nan")), dict(decay=float("inf")),
               dict(table=A, mp=1, page=32), dict(table=A, mp=0, page=64), dict(table=A, mp=4, page=0)):
        assert _attend(tq, **kw) == ARG, kw
    for kw in (dict(qd=9), dict(od=9), dict(Hq=18, bytes=1 << 30), dict(kcb=tq.tq_codebook_load(128, 8)),
               dict(vcb=tq.tq_codebook_load(128, 8)), dict(vcb=tq.tq_codebook_load(96, 2)),
               dict(table=A, mp=8, page=12), dict(table=A, mp=4, page=42)):
        assert _attend(tq, **kw) == UNSUPPORTED, kw
    for kw in (dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(work=ODD), dict(w=ODD), dict(lens=ODD),
               dict(table=ODD, mp=2, page=32), dict(q=P((1 << 20) + 1))):
        assert _attend(tq, **kw) == ALIGN, kw
    n = tq.tq_attn_weights_workspace_bytes(2, 8, 2, 50)
    assert _attend(tq, bytes=n - 1) == WORKSPACE
    assert _attend(tq, bytes=0) == WORKSPACE
    for bad in ((0, 8, 2, 50), (2, 7, 2, 50), (2, 18, 2, 50), (2, 8, 0, 50), (2, 8, 2, 0)):
        assert tq.tq_attn_weights_workspace_bytes(*bad) == 0
    # a score per token (in chunks of 32) and query head on top of the plain call's partials
    assert n >= tq.tq_attn_workspace_bytes_sms(2, 8, 2, 50, 1) - (1 << 20) and n >= 2 * 8 * 64 * 4


def _select(tq, **kw):
    a = dict(w=A, rs=100, lens=B, B=2, Hkv=2, T=100, keep=50, first=4, last=10, kept=C, new=D_)
    a.update(kw)
    return tq.lib().tq_evict_select(a["w"], a["rs"], a["lens"], a["B"], a["Hkv"], a["T"], a["keep"], a["first"],
                                    a["last"], a["kept"], a["new"], None)


def test_select_refusals(tq):
    for kw in (dict(w=None), dict(kept=None), dict(new=None), dict(B=0), dict(Hkv=0), dict(T=0), dict(keep=0),
               dict(first=-1), dict(last=-1), dict(first=45), dict(first=2**31 - 1, last=2**31 - 1), dict(rs=99),
               dict(lens=D_)):
        assert _select(tq, **kw) == ARG, kw
    for kw in (dict(w=ODD), dict(kept=ODD), dict(new=ODD), dict(lens=ODD)):
        assert _select(tq, **kw) == ALIGN, kw
    assert _select(tq, T=(1 << 30) + 1, rs=1 << 31) == UNSUPPORTED


def _compact(tq, **kw):
    a = dict(k=A, kb=66, v=B, vb=34, w=C, ws=100, kept=D_, keep=50, new=A, table=None, mp=0, page=0, np=0, B=2, Hkv=2,
             T_cap=104, T=100)
    a.update(kw)
    return tq.lib().tq_evict_compact(a["k"], a["kb"], a["v"], a["vb"], a["w"], a["ws"], a["kept"], a["keep"], a["new"],
                                     a["table"], a["mp"], a["page"], a["np"], a["B"], a["Hkv"], a["T_cap"], a["T"],
                                     None)


def test_compact_refusals(tq):
    for kw in (dict(k=None), dict(kept=None), dict(new=None), dict(B=0), dict(Hkv=0), dict(T=0), dict(keep=0),
               dict(kb=0), dict(vb=0), dict(ws=99), dict(T_cap=99), dict(table=B, mp=6, page=16, np=12),
               dict(table=B, mp=0, page=16, np=12), dict(table=B, mp=7, page=0, np=12),
               dict(table=B, mp=7, page=16, np=0)):
        assert _compact(tq, **kw) == ARG, kw
    for kw in (dict(kb=65), dict(vb=33), dict(k=P((1 << 20) + 1)), dict(kept=ODD), dict(new=ODD), dict(w=ODD),
               dict(table=ODD, mp=7, page=16, np=12)):
        assert _compact(tq, **kw) == ALIGN, kw
    for kw in (dict(kb=514), dict(vb=1 << 20), dict(T=(1 << 30) + 1, ws=1 << 31, T_cap=(1 << 30) + 8)):
        assert _compact(tq, **kw) == UNSUPPORTED, kw


def test_binding_refusals(tq):
    import torch
    x = torch.zeros(3, 2, 128)
    pos = torch.zeros(3, dtype=torch.int64)
    rope, cb = tq.tq_rope_load(), tq.tq_codebook_load(128, 4)
    with pytest.raises(ValueError, match="CUDA tensors"):
        tq.tq_rope_apply(x, pos, rope, x)
    for args in ((x[:, :, :64], pos, rope, x), (x, pos[:2], rope, x), (x, pos.int(), rope, x),
                 (x, pos[None].expand(2, 3), rope, x), (x, pos, rope, x[:, :1]), (x, pos, rope, x.half()),
                 (x.transpose(1, 2), pos, rope, x)):
        with pytest.raises(ValueError):
            tq.tq_rope_apply(*args)
    blocks = torch.zeros(8, 66, dtype=torch.uint8)
    dst = torch.arange(3)
    signs = tq.tq_signs()
    for k, v, kb, vb, d in ((None, None, None, None, dst), (x, None, None, None, dst), (x, x, blocks, blocks[:4], dst),
                            (x, x, blocks, blocks[:, :34], dst), (x, x[:2], blocks, blocks, dst),
                            (x, x.half(), blocks, blocks, dst), (x, x, blocks, blocks, dst.int()),
                            (x, x, blocks, blocks, dst[:2])):
        with pytest.raises(ValueError):
            tq.tq_insert_kv(k, v, pos, rope, cb, cb, signs, kb, vb, d, 4)
    with pytest.raises(ValueError):
        tq.tq_insert_kv(x, None, pos, rope, None, None, signs, blocks, None, dst, 4)
    q = torch.zeros(2, 8, 128)
    cache = torch.zeros(2, 2, 16, 66, dtype=torch.uint8)
    w = torch.zeros(2, 2, 16)
    lens = torch.zeros(2, dtype=torch.int32)
    ok = dict(q=q, k=cache, v=cache, w=w, out=q, T=10, lens=lens, table=None)
    for kw in (dict(q=q[:, :, :64]), dict(k=cache[:1]), dict(v=cache[:, :, :8].contiguous()), dict(w=w[:, :, :9]),
               dict(w=w.double()), dict(out=q[:1]), dict(lens=lens.long()), dict(table=torch.zeros(2, 2)),
               dict(w=w.transpose(0, 1)), dict()):
        a = dict(ok, **kw)
        with pytest.raises(ValueError):
            tq.tq_attn_decode_weights(a["q"], a["k"], cb, a["v"], cb, a["w"], a["out"], lens, a["T"], 0.1, signs,
                                      seq_lens=a["lens"], block_table=a["table"])
    kept = torch.zeros(2, 2, 4, dtype=torch.int32)
    for kw in (dict(kept=kept.long()), dict(new=lens[:1]), dict(new=None), dict(w=w[:1]), dict()):
        a = dict(dict(kept=kept, new=lens.clone(), w=w), **kw)
        with pytest.raises(ValueError):
            tq.tq_evict_select(a["w"], a["kept"], a["new"], 10, 1, 1, seq_lens=lens)
        with pytest.raises(ValueError):
            tq.tq_evict_compact(cache, cache, a["kept"], a["new"], 10, weights=a["w"])
    with pytest.raises(ValueError):
        tq.tq_evict_compact(cache, cache[:, :, :8].contiguous(), kept, lens, 10)
