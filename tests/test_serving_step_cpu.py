"""Argument checks of the page plan, the norms with rotary positions and the
shared-prefix attention, and their launches against the stand-in for the CUDA
runtime: host code only."""

import ctypes

import pytest

from test_launches_cpu import lib as _lib_copy, linked  # noqa: F401  (fixtures)
from test_rope_evict_cpu import ALIGN, ARG, ODD, UNSUPPORTED, WORKSPACE, A, B, C, D_, P, _bent, tq  # noqa: F401
from turboquant_bit_kv_gb300 import tq as real

E, F, G, H, I, J = (P(n << 20) for n in range(5, 11))
lib = _lib_copy


def _typed(fake):
    for name in ("tq_page_plan", "tq_norm_rope_apply", "tq_attn_decode_shared", "tq_attn_shared_workspace_bytes"):
        getattr(fake, name).argtypes = getattr(real.lib(), name).argtypes
        getattr(fake, name).restype = getattr(real.lib(), name).restype
    return fake


def _plan(L, **kw):
    a = dict(cached=A, fresh=B, start=None, B=4, Hkv=2, page=16, table=C, row=10, most=10, held=D_, nheld=D_, free=E,
             nfree=100, count=F, ncount=F, seq=G, tok=H, dst=I, pos=J, n=64)
    a.update(kw)
    return L.tq_page_plan(a["cached"], a["fresh"], a["start"], a["B"], a["Hkv"], a["page"], a["table"], a["row"],
                          a["most"], a["held"], a["nheld"], a["free"], a["nfree"], a["count"], a["ncount"], a["seq"],
                          a["tok"], a["dst"], a["pos"], a["n"], None)


PLAN_BAD = [(ARG, kw) for kw in (
    dict(cached=None), dict(fresh=None), dict(table=None), dict(held=None), dict(nheld=None), dict(free=None),
    dict(count=None), dict(ncount=None), dict(seq=None), dict(tok=None), dict(dst=None), dict(pos=None), dict(B=0),
    dict(Hkv=0), dict(page=0), dict(most=0), dict(nfree=-1), dict(n=-1), dict(row=9), dict(row=-1), dict(seq=A), dict(tok=B),
    dict(table=D_), dict(dst=E), dict(pos=F), dict(start=J),
    dict(nheld=A), dict(nheld=F), dict(ncount=B), dict(ncount=D_), dict(ncount=E))] + [(ALIGN, kw) for kw in (
        dict(cached=ODD), dict(fresh=ODD), dict(table=ODD), dict(held=ODD), dict(nheld=ODD), dict(free=ODD),
        dict(count=ODD), dict(ncount=ODD), dict(seq=ODD), dict(tok=ODD), dict(dst=ODD), dict(pos=ODD),
        dict(start=ODD))] + [(UNSUPPORTED, kw) for kw in (dict(n=1 << 31), dict(B=(1 << 24) + 1))]


@pytest.mark.parametrize("want,kw", PLAN_BAD)
def test_plan_refusals(lib, want, kw):  # noqa: F811
    L = _typed(lib)
    assert _plan(L, **kw) == want
    assert L.fake_launches() == 0


def test_plan_launches(lib):  # noqa: F811
    L = _typed(lib)
    for kw, n in ((dict(), 1), (dict(n=0, dst=None, pos=None), 1), (dict(nfree=0, free=None), 1), (dict(n=100000), 2), (dict(n=100000, nheld=P(11 << 20)), 2),
                  (dict(n=100000, ncount=P(11 << 20)), 2),
                  (dict(n=100000, nheld=P(11 << 20), ncount=P(12 << 20)), 1),
                  (dict(B=1, row=0), 1), (dict(nheld=I, dst=D_, held=J, pos=C, table=A, cached=H, tok=E, free=G, seq=B,
                                               fresh=F, count=P(11 << 20), ncount=P(12 << 20)), 1)):
        L.fake_reset()
        assert _plan(L, **kw) == 0, kw
        assert L.fake_launches() == n
        for i in range(1, n + 1):
            L.fake_fail_at(i)
            assert _plan(L, **kw) == real.TQ_ERR_CUDA
            L.fake_fail_at(0)
            assert _plan(L, **kw) == 0


def _norm(L, **kw):
    a = dict(q=A, qh=4, qt=1024, qs=128, k=B, kh=2, kt=1024, ks=128, dtype=real.TQ_BF16, n=4, qw=C, kw=D_,
             wd=real.TQ_BF16, eps=1e-6, pos=E, pa=4, rope=real.tq_rope_load(), qo=F, qot=512, qos=128, ko=G, kot=256,
             kos=128)
    a.update(kw)
    r = a["rope"]
    return L.tq_norm_rope_apply(a["q"], a["qh"], a["qt"], a["qs"], a["k"], a["kh"], a["kt"], a["ks"], a["dtype"], a["n"],
                                a["qw"], a["kw"], a["wd"], a["eps"], a["pos"], a["pa"],
                                None if r is None else ctypes.byref(r), a["qo"], a["qot"], a["qos"], a["ko"], a["kot"],
                                a["kos"], None)


def test_norm_refusals(lib):  # noqa: F811
    L = _typed(lib)
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(n=-1), dict(qh=-1),
               dict(qh=0, kh=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(qt=-1024), dict(ks=-128), dict(pa=-1), dict(qot=384), dict(kos=64)):
        assert _norm(L, **kw) == ARG, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(qo=ODD), dict(ko=ODD), dict(qt=1028), dict(kos=132), dict(pos=P((1 << 20) + 4)),
               dict(qw=P((1 << 20) + 1)), dict(kw=P((1 << 20) + 1))):
        assert _norm(L, **kw) == ALIGN, kw
    for kw in (dict(dtype=9), dict(wd=9), dict(rope=_bent(real, rot_dim=40)), dict(qh=1 << 26, kh=1 << 26)):
        assert _norm(L, **kw) == UNSUPPORTED, kw
    assert L.fake_launches() == 0
    assert _norm(L, n=0) == 0 and L.fake_launches() == 0
    for kw in (dict(), dict(qh=0, q=None, qo=None), dict(kh=0, k=None, ko=None), dict(rope=None, pos=None),
               dict(qw=None, kw=None), dict(qo=A, qot=1024), dict(n=20000)):
        L.fake_reset()
        assert _norm(L, **kw) == 0 and L.fake_launches() == 1, kw
    L.fake_fail_at(1)
    assert _norm(L) == real.TQ_ERR_CUDA
    L.fake_fail_at(0)
    assert _norm(L) == 0


def _shared(L, **kw):
    a = dict(q=A, qd=real.TQ_BF16, kp=B, vp=C, pt=None, P_cap=1024, P=1000, pl=None, k=D_, kcb=real.tq_codebook_load(128, 4),
             v=E, vcb=real.tq_codebook_load(128, 2), table=None, row=0, mp=0, page=0, lens=None, B=2, Hq=8, Hkv=2,
             T_cap=64, T=50, scale=0.1, out=F, od=real.TQ_F32, ws=G, bytes=None)
    a.update(kw)
    n = L.tq_attn_shared_workspace_bytes(a["B"], a["Hq"], a["Hkv"], a["P"], a["T"]) if a["bytes"] is None else a["bytes"]
    ref = {m: None if a[m] is None else ctypes.byref(a[m]) for m in ("kcb", "vcb")}
    return L.tq_attn_decode_shared(a["q"], a["qd"], a["kp"], a["vp"], a["pt"], a["P_cap"], a["P"], a["pl"], a["k"],
                                   ref["kcb"], a["v"], ref["vcb"], a["table"], a["row"], a["mp"], a["page"], a["lens"],
                                   a["B"], a["Hq"], a["Hkv"], a["T_cap"], a["T"], a["scale"], real.tq_signs(), a["out"],
                                   a["od"], a["ws"], n, None)


def test_shared_refusals(lib):  # noqa: F811
    L = _typed(lib)
    paged = dict(table=H, pt=I, row=4, mp=4, page=16, P_cap=1008)
    for kw in (dict(q=None), dict(kp=None), dict(vp=None), dict(k=None), dict(v=None), dict(kcb=None), dict(vcb=None),
               dict(out=None), dict(ws=None), dict(B=0), dict(Hq=7), dict(Hkv=0), dict(T=0), dict(P=0), dict(P=1025),
               dict(P_cap=1004), dict(T=65), dict(T_cap=60), dict(scale=float("nan")), dict(pt=I), dict(table=H, page=16),
               dict(paged, mp=3), dict(paged, row=3), dict(paged, page=0), dict(paged, mp=0), dict(paged, P=1009),
               dict(paged, row=1 << 31)):
        assert _shared(L, **kw) == ARG, kw
    bent = real.tq_codebook_load(128, 4)
    bent.centroids[3] *= 1.5
    for kw in (dict(qd=9), dict(od=9), dict(Hq=18, bytes=1 << 30), dict(kcb=real.tq_codebook_load(128, 8)),
               dict(vcb=real.tq_codebook_load(64, 4)), dict(paged, page=20), dict(vcb=bent),
               dict(P=(1 << 31) - 8191, P_cap=(1 << 31) - 8, bytes=1 << 62)):
        assert _shared(L, **kw) == UNSUPPORTED, kw
    for kw in (dict(kp=ODD), dict(vp=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(ws=ODD), dict(lens=ODD),
               dict(pl=ODD), dict(paged, table=ODD), dict(paged, pt=ODD), dict(q=P((1 << 20) + 1))):
        assert _shared(L, **kw) == ALIGN, kw
    n = L.tq_attn_shared_workspace_bytes(2, 8, 2, 1000, 50)
    assert n > 0 and _shared(L, bytes=n - 1) == WORKSPACE and _shared(L, bytes=0) == WORKSPACE
    for bad in ((0, 8, 2, 9, 9), (2, 7, 2, 9, 9), (2, 18, 2, 9, 9), (2, 8, 2, 0, 9), (2, 8, 2, 9, 0), (2, 8, 2, 1 << 31, 9)):
        assert L.tq_attn_shared_workspace_bytes(*[min(x, 2**31 - 1) for x in bad]) == 0
    assert L.fake_launches() == 0
    for kb in (2, 3, 4):
        for vb in (2, 3, 4):
            for kw in (dict(), paged, dict(B=100, Hq=16)):
                L.fake_reset()
                cbs = dict(kcb=real.tq_codebook_load(128, kb), vcb=real.tq_codebook_load(128, vb))
                assert _shared(L, **kw, **cbs) == 0 and L.fake_launches() == 4, (kb, vb, kw)
    for i in range(1, 5):
        L.fake_fail_at(i)
        assert _shared(L) == real.TQ_ERR_CUDA and L.fake_launches() == i
        L.fake_fail_at(0)
        assert _shared(L) == 0


@pytest.mark.parametrize("B,Hq,Hkv", [(1, 32, 8), (64, 56, 8), (200, 16, 2), (5, 8, 1), (33, 64, 8)])
def test_shared_workspace_holds_shorter(lib, B, Hq, Hkv):  # noqa: F811
    """A workspace for P and T tokens is one for fewer, at every number of tiles (the work is cut otherwise for each)."""
    L = _typed(lib)
    last = 0
    for P in (1, 128, *range(129, 90000, 128), 10**6, 2**31 - 8192):
        n = L.tq_attn_shared_workspace_bytes(B, Hq, Hkv, P, 100)
        assert n >= last, P
        last = n
    assert _shared(L, B=B, Hq=Hq, Hkv=Hkv, P=20 * 128 + 1, P_cap=20 * 128 + 8,
                   bytes=L.tq_attn_shared_workspace_bytes(B, Hq, Hkv, 21 * 128 + 1, 50)) == 0
    last = 0
    for T in (1, 31, 32, 33, 1000, 5000, 10**6, 2**31 - 8192):
        n = L.tq_attn_shared_workspace_bytes(B, Hq, Hkv, 1000, T)
        if B * Hkv * -(-T // 32) > 2**31 - 1:   # pieces of 32 tokens are counted in 31 bits: refused
            assert n == 0
            continue
        assert n >= last, T
        last = n


def test_binding_refusals(tq):  # noqa: F811
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    one, tok, table = i[:1].clone(), torch.zeros(5, dtype=torch.int32), torch.zeros(4, 6, dtype=torch.int32)
    long = torch.zeros(9, dtype=torch.int64)
    ok = dict(cached=i, fresh=i, held=i, table=table, free=i, count=one, nheld=i, ncount=one, seq=i, tok=tok, dst=long,
              pos=long, start=None)
    for kw in (dict(cached=i[:3]), dict(fresh=i.long()), dict(held=i[::2]), dict(table=table.long()), dict(table=table.T),
               dict(count=i), dict(tok=i), dict(dst=long.int()), dict(pos=long[:5]), dict(start=i), dict(seq=i[:2]),
               dict(free=table), dict()):
        a = dict(ok, **kw)
        with pytest.raises(ValueError):
            tq.tq_page_plan(a["cached"], a["fresh"], a["held"], a["table"], a["free"], a["count"], 16, 2, a["nheld"],
                            a["ncount"], a["seq"], a["tok"], a["dst"], a["pos"], pos_start=a["start"])
    x, w, pos, rope = torch.zeros(3, 2, 128), torch.ones(128), torch.zeros(3, dtype=torch.int64), tq.tq_rope_load()
    for args in ((None, None, None, None, 1e-6, pos, rope, None, None), (x, None, w, None, 1e-6, pos, rope, None, None),
                 (x, x, w, w, 1e-6, pos, rope, x, None), (x, x[:2], w, w, 1e-6, pos, rope, x, x[:2]),
                 (x, x.half(), w, w, 1e-6, pos, rope, x, x.half()), (x, x, w[:64], w, 1e-6, pos, rope, x, x),
                 (x, x, w, w.half(), 1e-6, pos, rope, x, x), (x, x, w, w, 1e-6, pos[:2], rope, x, x),
                 (x, x, w, w, 1e-6, pos, rope, x[:, :1], x), (x[..., :64], x, w, w, 1e-6, pos, rope, x, x),
                 (x, x, w, w, 1e-6, pos, rope, x, x)):
        with pytest.raises(ValueError):
            tq.tq_norm_rope_apply(*args)
    q, cb, signs = torch.zeros(2, 8, 128), tq.tq_codebook_load(128, 4), tq.tq_signs()
    pre, own = torch.zeros(2, 16, 66, dtype=torch.uint8), torch.zeros(2, 2, 16, 66, dtype=torch.uint8)
    lens, t1, t2 = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    ok = dict(q=q, kp=pre, vp=pre, k=own, v=own, out=q, pl=None, pt=None, lens=lens, table=None)
    pg = dict(kp=own, vp=own, pt=t1, table=t2)
    for kw in (dict(q=q[..., :64]), dict(kp=pre[:1]), dict(vp=pre[..., :34]), dict(k=own[:1]), dict(v=own[:, :, :8]),
               dict(out=q[:1]), dict(pl=lens), dict(lens=lens.long()), dict(pt=t1), dict(table=t2), dict(pg, pt=t2),
               dict(pg, table=t2.long()), dict(pg, table=t2[:1]), dict(pg, kp=pre), dict(pg, vp=own[..., :34]), dict(pg),
               dict()):
        a = dict(ok, **kw)
        with pytest.raises(ValueError):
            tq.tq_attn_decode_shared(a["q"], a["kp"], a["vp"], a["k"], cb, a["v"], cb, a["out"], lens, 10, 10, 0.1, signs,
                                     prefix_len=a["pl"], prefix_table=a["pt"], seq_lens=a["lens"], block_table=a["table"])
