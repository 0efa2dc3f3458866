"""Page plan, norms with rotary positions and shared-prefix attention against
plain computations, and a serving loop of all of them.

Tolerances.  Page plan: whole numbers, equal to a loop over the requests.

Norms: the sum of 128 squares is off by 19 roundings at most (16 in a thread, 3
between threads), of which the root halves the effect; the root itself is good
to 2 ulp, its products with the element and the weight are a rounding each:
(19 / 2 + 4 + 2) 2^-24 < 2^-20 of the element.  The rotation adds 2^-22 (|a| +
|b|) and the output type eps / 2 of the value.

Attention.  As for the decode attention with weights: with S = sum_t p_t ||v_t||
of a query head, scores off by ds, outputs by (2 ds + 2^-17 + eps_v) S plus the
output type's rounding.  Behind a prefix the keys' levels are fp16 under a common
factor, off by eps_k = 2^-18 / 2^-15 / 2^-13.5 (2 / 3 / 4 bits) of each at most,
and so are the values': ds = scale ||q|| ||k|| (eps_k + 2^-21 + 2^-18) + ||k|| (12 + 12
scale ||q||) 2^-25."""

import numpy as np
import pytest
import torch

import oracle
from oracle import codec
from parity_util import oracle_books
from test_gpu_evict import cache_of
from test_gpu_rope_insert import ROPES, rotated
from turboquant_bit_kv_gb300 import workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE = 1 / np.sqrt(128)
LEVEL_EPS = {2: 2.0**-18, 3: 2.0**-15, 4: 2.0**-13.5}


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from turboquant_bit_kv_gb300 import tq as mod
    mod.lib()
    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- page plan

def plan_reference(cached, fresh, held, table, free, count, page, Hkv, n_tok, start):
    B, most = table.shape
    table, held = table.copy(), np.clip(held, 0, most)
    count = min(max(count, 0), len(free))
    seq, tok = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    dst, pos = np.full(n_tok, -1, np.int64), np.zeros(n_tok, np.int64)
    open_ = True
    for b in range(B):
        c, m = max(int(cached[b]), 0), max(int(fresh[b]), 0)
        tok[b + 1] = tok[b] + m
        fits = c + m <= min(most * page, 2**31 - 1) and tok[b + 1] <= n_tok
        need = max(0, -(-(c + m) // page) - int(held[b])) if fits and m else 0
        if need and need > count:
            open_ = False
        ok = fits and (need == 0 or open_)
        if ok and need:
            for i in range(need):
                count -= 1
                table[b, held[b] + i] = free[count]
            held[b] += need
        seq[b] = c + m if ok else c
        for i in range(min(m, n_tok - int(tok[b])) if tok[b] < n_tok else 0):
            t = c + i
            pos[tok[b] + i] = (c if start is None else int(start[b])) + i
            if ok:
                dst[tok[b] + i] = int(table[b, t // page]) * Hkv * page + t % page
    return table, held, count, seq, np.minimum(tok, 2**31 - 1), dst, pos


def plan_call(tq, cached, fresh, held, table, free, count, page, Hkv, n_tok, start, in_place=False, stride=0):
    B, most = table.shape
    wide = torch.full((B, most + stride), -7, dtype=torch.int32, device="cuda")
    view = wide[:, :most]
    view.copy_(i32(table))
    h, c = i32(held), i32([count])
    nh, nc = (h, c) if in_place else (torch.empty_like(h), torch.empty_like(c))
    seq, tok = torch.empty_like(h), torch.empty(B + 1, dtype=torch.int32, device="cuda")
    dst = torch.full((n_tok,), -99, dtype=torch.int64, device="cuda")
    pos = torch.full((n_tok,), -99, dtype=torch.int64, device="cuda")
    s = None if start is None else torch.tensor(start, device="cuda")
    args = (i32(cached), i32(fresh), h, view, i32(free), c, page, Hkv, nh, nc, seq, tok, dst, pos)
    tq.tq_page_plan(*args, pos_start=s)
    assert torch.all(wide[:, most:] == -7)
    return [x.cpu().numpy() for x in (view, nh, nc[0], seq, tok, dst, pos)]


def same_plan(got, want):
    for name, g, w in zip(("table", "held", "count", "seq_lens", "tok_start", "dst", "pos"), got, want):
        assert np.array_equal(g, w), (name, np.argwhere(np.asarray(g) != np.asarray(w))[:4])


@pytest.mark.parametrize("B,page,short,most_new", [
    (1, 16, 0, 1), (1, 8, 0, 0), (3, 64, 0, 200), (33, 16, 0, 40), (64, 1, 0, 3), (64, 16, 1, 40), (300, 100, 2, 30),
    (1023, 8, 0, 5), (1024, 8, 1, 5), (1025, 8, 1, 5), (2500, 16, 0, 4), (2500, 16, 1, 4), (7, 16, 0, 3000),
    (40, 32, 1, 900)])
def test_page_plan(tq, B, page, short, most_new):
    rng = np.random.default_rng(B * 1000 + page + short)
    cached = rng.integers(0, 5 * page + 1, B)
    fresh = rng.integers(0, most_new + 1, B)
    fresh[rng.random(B) < 0.2] = 0
    cached[rng.random(B) < 0.1] = -3                            # (taken as 0)
    fresh[rng.random(B) < 0.05] = -2
    most = int((cached.clip(0) + fresh.clip(0)).max()) // page + 2
    held = -(-cached.clip(0) // page)
    held = np.where(rng.random(B) < 0.2, held + rng.integers(0, 2, B), held)     # pages ahead
    if B > 4:
        cached[4], fresh[4] = most * page - 1, 2                # more than a row holds: refused
        held[4] = most
    ids = rng.permutation(4 * B * most + 10)
    table = np.full((B, most), -1)
    for b in range(B):
        table[b, :held[b]] = ids[b * most:b * most + held[b]]
    free = ids[B * most:]
    need = int(np.maximum(0, -(-(cached.clip(0) + fresh.clip(0)) // page) - held)[fresh > 0].sum())
    count = {0: min(len(free), need + 5), 1: need // 2, 2: 0}[short]
    total = int(fresh.clip(0).sum())
    start = cached + rng.integers(0, 1000, B) * 1000003 if B % 2 else None
    for n_tok in sorted({total, total + 37, max(0, total - 5), 0}):
        want = plan_reference(cached, fresh, held, table, free, count, page, 3, n_tok, start)
        for kw in (dict(), dict(in_place=True, stride=5)):
            got = plan_call(tq, cached, fresh, held, table, free, count, page, 3, n_tok, start, **kw)
            same_plan(got, want)


def test_page_plan_large(tq):
    """The tokens' own grid, and sums past 32 bits."""
    B, page = 40, 16
    cached, fresh = np.arange(B) * 7, np.full(B, 3001)
    most = 3300 // page + 1
    held = -(-cached // page)
    table = np.where(np.arange(most) < held[:, None], np.arange(B * most).reshape(B, most), -1)
    free = np.arange(B * most, 3 * B * most)
    want = plan_reference(cached, fresh, held, table, free, len(free), page, 8, 3001 * B + 700, None)
    same_plan(plan_call(tq, cached, fresh, held, table, free, len(free), page, 8, 3001 * B + 700, None), want)
    cached, fresh = np.array([2**31 - 1, 5, 2**31 - 10, 0]), np.array([2**31 - 1, 2**31 - 1, 2, 2**31 - 1])
    table = np.arange(40).reshape(4, 10)
    got = plan_call(tq, cached, fresh, [10, 1, 10, 1], table, free, 7, page, 8, 5000, None)
    assert got[3].tolist() == [2**31 - 1, 5, 2**31 - 10, 0] and got[2] == 7 and np.array_equal(got[0], table)
    assert got[4].tolist() == [0, 2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1]
    assert np.all(got[5] == -1) and np.array_equal(got[6], 2**31 - 1 + np.arange(5000))
    got = plan_call(tq, [4], [4], [5], np.arange(10).reshape(1, 10), [], 0, page, 8, 4, None)   # no free page at all
    assert got[3].tolist() == [8] and got[5].tolist() == [4, 5, 6, 7]


@pytest.mark.parametrize("most_new", [3, 2000])
def test_page_plan_holds_fewer_than_cached(tq, most_new):
    """Requests that hold fewer pages than their cached tokens fill take those too; requests that hold more than their
    row has are taken to hold its pages."""
    rng = np.random.default_rng(most_new)
    B, page = 30, 16
    cached, fresh = rng.integers(0, 200, B), rng.integers(0, most_new + 1, B)
    most = (200 + most_new) // page + 2
    held = rng.integers(0, -(-cached // page) + 1)
    held[3], held[4] = most + 5, -2
    ids = rng.permutation(3 * B * most)
    table = np.where(np.arange(most) < held[:, None], ids[:B * most].reshape(B, most), -1)
    total = int(fresh.sum())
    for count in (2 * B * most, 40):
        args = (cached, fresh, held, table, ids[B * most:], count, page, 2, total + 9, None)
        same_plan(plan_call(tq, *args), plan_reference(*args))
        same_plan(plan_call(tq, *args, in_place=True, stride=1), plan_reference(*args))


def test_page_plan_far_pages(tq):
    """Page numbers whose slots pass 32 bits."""
    top = 2**31 - 1
    cached, fresh, page, Hkv = np.array([5, 0]), np.array([200, 3]), 128, 8
    table = np.full((2, 3), -1)
    table[0, 0] = top
    free = np.array([7, top - 1, top - 2])
    want = plan_reference(cached, fresh, np.array([1, 0]), table, free, 3, page, Hkv, 203, None)
    assert want[5].max() > 2**40
    same_plan(plan_call(tq, cached, fresh, [1, 0], table, free, 3, page, Hkv, 203, None), want)


# ---------------------------------------------------------------- norms with rotary positions

def norm_reference(x, w, eps, pos, rope):
    """float64 [n, heads, 128] -> normalised and turned, and its tolerance before the output type's rounding."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if rope is None:
        return y, 2.0**-20 * np.abs(y)
    out, size = rotated(y, pos, rope)
    return out, np.where(size > 0, 2.0**-22 * size + 2.0**-20 * size, 2.0**-20 * np.abs(y))


def check_norm(out, want, tol, dtype):
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * eps * 2
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= eps * np.abs(want) + tol * (1 + eps) + tiny), (err / (np.abs(want) + 1e-30)).max()


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f16"), ("f32", None)])
@pytest.mark.parametrize("kw", ROPES[:8:1] + [None])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (7, 5, 1), (130, 28, 4), (700, 3, 3)])
def test_norm_rope(tq, dtype, wdtype, kw, n, hq, hkv):
    rope = None if kw is None else tq.tq_rope_load(**kw)
    g = torch.Generator(device="cuda").manual_seed(n * 100 + hq)
    buf = (torch.randn(n, hq + 2 * hkv + 1, 128, generator=g, device="cuda") *
           torch.exp(2 * torch.randn(n, hq + 2 * hkv + 1, 1, generator=g, device="cuda"))).to(DT[dtype])
    q, k = buf[:, :hq], buf[:, hq:hq + hkv]                     # strided rows of one projection
    w = [None, None] if wdtype is None else [
        (1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(DT[wdtype]) for _ in range(2)]
    pos = None if rope is None else torch.randint(-2**40, 2**62, (rope.axes, n), generator=g, device="cuda")
    qo = torch.full((n, hq + 1, 128), 7.0, dtype=DT[dtype], device="cuda")
    ko = torch.full((n, hkv, 128), 7.0, dtype=DT[dtype], device="cuda")
    before = buf.clone()
    tq.tq_norm_rope_apply(q, k, w[0], w[1], 1e-6, pos, rope, qo[:, :hq], ko)
    assert torch.equal(buf, before) and torch.all(qo[:, hq] == 7.0)
    eps = float(np.float32(1e-6))
    for x, wi, out in ((q, w[0], qo[:, :hq]), (k, w[1], ko)):
        wi = 1.0 if wi is None else wi.double().cpu().numpy()
        want, tol = norm_reference(x.double().cpu().numpy(), wi, eps, None if pos is None else pos.cpu().numpy(), rope)
        check_norm(out, want, tol, DT[dtype])
    # one of them alone, and in place
    ko2 = torch.empty_like(ko)
    tq.tq_norm_rope_apply(None, k, None, w[1], 1e-6, pos, rope, None, ko2)
    assert torch.equal(ko2, ko)
    tq.tq_norm_rope_apply(q, k, w[0], w[1], 1e-6, pos, rope, q, k)
    assert torch.equal(q, qo[:, :hq]) and torch.equal(k, ko)
    assert torch.equal(buf[:, hq + hkv:], before[:, hq + hkv:])


def test_norm_rope_far_rows(tq):
    """Rows past 2^32 bytes and 2^31 elements."""
    n, hq, hkv = 140000, 112, 16
    x = torch.empty(n, hq + hkv, 128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.tensor([0, 1, 65535, 131071, 139999], device="cuda")
    x.fill_(1.0)
    x[rows] = torch.randn(5, hq + hkv, 128, generator=g, device="cuda").bfloat16()
    pos = torch.arange(n, device="cuda")
    rope = tq.tq_rope_load()
    qo, ko = torch.empty(n, hq, 128, dtype=x.dtype, device="cuda"), torch.empty(n, hkv, 128, dtype=x.dtype, device="cuda")
    tq.tq_norm_rope_apply(x[:, :hq], x[:, hq:], None, None, 1e-6, pos, rope, qo, ko)
    want, tol = norm_reference(x[rows].double().cpu().numpy(), 1.0, float(np.float32(1e-6)), pos[rows][None].cpu().numpy(), rope)
    check_norm(torch.cat([qo[rows], ko[rows]], 1), want, tol, x.dtype)


def test_norm_rope_ranges(tq):
    """Zero rows, tiny and huge elements, infinities and NaN."""
    x = torch.ones(8, 1, 128, device="cuda")
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 3e38                                               # squares past float32
    x[3] *= 1e19
    x[4, 0, 5], x[5, 0, 7] = float("inf"), float("nan")
    x[6, 0, 100] = 3e38
    x[7] *= 2e17                                               # the sum, not the squares
    out = torch.empty_like(x)
    tq.tq_norm_rope_apply(x, None, None, None, 1e-6, None, None, out, None)
    y = out[:, 0].double().cpu().numpy()
    eps = float(np.float32(1e-6))
    ref = x[:, 0].double().cpu().numpy()
    want = ref / np.sqrt((ref**2).mean(-1, keepdims=True) + eps)
    for i in (0, 1, 2, 3, 6, 7):
        assert np.all(np.abs(y[i] - want[i]) <= 2.0**-20 * np.abs(want[i]) + 2.0**-126), i
    assert np.isnan(y[4, 5]) and np.all(np.delete(y[4], 5) == 0)
    assert np.isnan(y[5]).all()


# ---------------------------------------------------------------- attention behind a shared prefix

def attend_reference(q, kp, vp, ko, vo, lens, kb, vb, scale=SCALE, eps_v=None):
    """q [B, Hq, 128], prefix [Hkv, P, 128], own [B, Hkv, T, 128] -> out and its tolerance."""
    B, Hq, _ = q.shape
    Hkv = kp.shape[0]
    G = Hq // Hkv
    out, tol = np.zeros((B, Hq, 128)), np.zeros((B, Hq, 1))
    for b in range(B):
        if lens[b] < 0 or kp.shape[1] + lens[b] == 0:
            continue
        for h in range(Hkv):
            k = np.concatenate([kp[h], ko[b, h, :lens[b]]])
            v = np.concatenate([vp[h], vo[b, h, :lens[b]]])
            x = q[b, h * G:(h + 1) * G]
            s = scale * x @ k.T
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[b, h * G:(h + 1) * G] = p @ v
            # each score's own error, on the keys that carry weight: |o| moves by sum p (err_t + mean err) ||v||
            qn, kn, vn = np.linalg.norm(x, axis=-1, keepdims=True), np.linalg.norm(k, axis=-1), np.linalg.norm(v, axis=-1)
            ds = scale * qn * kn * (LEVEL_EPS[kb] + 2.0**-21 + 2.0**-18) + kn * (12 + 12 * scale * qn) * 2.0**-25
            S = (p * vn).sum(-1)
            mean = (p * ds).sum(-1)
            tol[b, h * G:(h + 1) * G, 0] = (p * np.expm1(2 * ds) * vn).sum(-1) + 2 * mean * S + \
                (2.0**-17 + (eps_v or LEVEL_EPS[vb])) * S
    return out, tol


class Case:
    """A batch behind a prefix: contiguous caches, or pools with tables, garbage in every slot that holds no token."""

    def __init__(self, B, Hq, Hkv, P, T, kb, vb, page, lens, qd="bf16", seed=0, loud=1.0, q_size=1.0, slack=0):
        rng = np.random.default_rng(seed)
        self.shape, self.bits, self.lens = (B, Hq, Hkv, P, T), (kb, vb), lens
        self.eff = [T] * B if lens is None else [min(n, T) for n in lens]
        self.bound = P + slack
        (kp, self.kp), (vp, self.vp) = (cache_of((Hkv, P), b, rng, loud) for b in (kb, vb))
        (ko, self.ko), (vo, self.vo) = (cache_of((B, Hkv, T), b, rng, loud) for b in (kb, vb))
        self.q = (torch.from_numpy(rng.standard_normal((B, Hq, 128))) * q_size).to(DT[qd])
        self.prefix_table = self.table = None

        def garbage(shape):
            x = rng.integers(0, 256, shape, dtype=np.uint8)
            x[..., 0], x[..., 1] = 0xFF, 0x7F                  # norms that are NaN
            return x

        if page:
            np_, no = -(-self.bound // page), -(-T // page)
            used = -(-P // page)
            ids = rng.permutation(np_ + B * no + 3)
            table = np.full((B, np_ + no + 2), -1)
            table[:, :used] = ids[:used]                       # entries behind the prefix's tokens name nothing
            for b in range(B):
                n = -(-max(self.eff[b], 0) // page)
                table[b, np_:np_ + n] = ids[np_ + b * no:np_ + b * no + n]
            self.full = i32(table)
            self.prefix_table, self.table = self.full[0, :np_], self.full[:, np_:]
            pools = []
            for pre, own in ((kp, ko), (vp, vo)):
                pool = garbage((len(ids), Hkv, page, pre.shape[-1]))
                for i in range(used):
                    part = pre[:, i * page:(i + 1) * page]
                    pool[ids[i], :, :part.shape[1]] = part
                for b in range(B):
                    for i in range(-(-max(self.eff[b], 0) // page)):
                        part = own[b, :, i * page:min((i + 1) * page, self.eff[b])]
                        pool[table[b, np_ + i], :, :part.shape[1]] = part
                pools.append(torch.from_numpy(pool).cuda())
            self.k = self.k_prefix = pools[0]
            self.v = self.v_prefix = pools[1]
        else:
            cap = (T + 7) // 8 * 8 + 8
            pcap = (self.bound + 7) // 8 * 8 + 8
            for name, pre, own in (("k", kp, ko), ("v", vp, vo)):
                full = garbage((Hkv, pcap, pre.shape[-1]))
                full[:, :P] = pre
                setattr(self, name + "_prefix", torch.from_numpy(full).cuda())
                full = garbage((B, Hkv, cap, own.shape[-1]))
                for b in range(B):
                    full[b, :, :max(self.eff[b], 0)] = own[b, :, :max(self.eff[b], 0)]
                setattr(self, name, torch.from_numpy(full).cuda())
        self.prefix_len = i32([P]) if slack else None

    def args(self, tq, od, ws=None):
        B, Hq, Hkv, P, T = self.shape
        out = torch.full((B, Hq, 128), float("nan"), dtype=DT[od], device="cuda")
        if ws is None:
            n = tq.tq_attn_shared_workspace_bytes(B, Hq, Hkv, self.bound, T)
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        kcb, vcb = (tq.tq_codebook_load(128, b) for b in self.bits)
        a = (self.q.cuda(), self.k_prefix, self.v_prefix, self.k, kcb, self.v, vcb, out, ws, self.bound, T, SCALE,
             tq.tq_signs_from_seed(workloads.SIGN_SEED))
        kw = dict(prefix_len=self.prefix_len, prefix_table=self.prefix_table,
                  seq_lens=None if self.lens is None else i32(self.lens), block_table=self.table)
        return a, kw, out

    def check(self, out, ref=None):
        want, tol = ref or attend_reference(self.q.double().numpy(), self.kp, self.vp, self.ko, self.vo, self.eff,
                                            *self.bits)
        eps = torch.finfo(out.dtype).eps / 2
        got = out.double().cpu().numpy()
        gone = ~np.isfinite(want).all(-1)                      # norms past fp16: infinite blocks, and no finite output
        assert not np.isfinite(got[gone]).any()
        if not gone.all():
            g, w, t = got[~gone], want[~gone], tol[~gone]
            over = np.abs(g - w) / (t * (1 + eps) + eps * np.abs(w) + 1e-37)
            assert np.isfinite(over).all() and over.max() <= 1, (over.max(), np.unravel_index(np.nanargmax(over), over.shape))
        return want, tol


def run_shared(tq, *a, od="f32", **kw):
    c = Case(*a, **kw)
    args, kws, out = c.args(tq, od)
    tq.tq_attn_decode_shared(*args, **kws)
    c.check(out)
    assert tq.tq_device_status() == tq.TQ_OK
    again = c.args(tq, od)
    tq.tq_attn_decode_shared(*again[0], **again[1])
    assert torch.equal(again[2].nan_to_num(7.0), out.nan_to_num(7.0))      # the same bits
    return c, out


@pytest.mark.parametrize("kb", [2, 3, 4])
@pytest.mark.parametrize("vb", [2, 3, 4])
def test_shared_formats(tq, kb, vb):
    run_shared(tq, 3, 8, 2, 300, 77, kb, vb, 0, [77, 0, 12], seed=kb * 10 + vb)
    run_shared(tq, 40, 14, 2, 300, 40, kb, vb, 16, [40 - b for b in range(40)], seed=kb * 10 + vb, qd="f16", od="f16")


def test_shared_far_pages(tq):
    """Pools past 2^32 bytes, the pages in use at their end."""
    c = Case(5, 8, 1, 300, 70, 4, 4, 64, [70, 0, 64, 3, 33], seed=77, qd="f32")
    far = 1100000
    pools = []
    for pool in (c.k, c.v):
        big = torch.empty(far + pool.shape[0], *pool.shape[1:], dtype=torch.uint8, device="cuda")
        assert big.numel() > 2**32
        big[far:] = pool
        pools.append(big)
    c.k = c.k_prefix = pools[0]
    c.v = c.v_prefix = pools[1]
    np_ = c.prefix_table.numel()
    c.full = torch.where(c.full >= 0, c.full + far, c.full)
    c.prefix_table, c.table = c.full[0, :np_], c.full[:, np_:]
    args, kw, out = c.args(tq, "f32")
    tq.tq_attn_decode_shared(*args, **kw)
    c.check(out)


@pytest.mark.parametrize("P", [1, 7, 8, 127, 128, 129, 255, 256, 257, 1000, 4133])
@pytest.mark.parametrize("B,G", [(1, 1), (5, 8), (37, 7), (50, 6)])
def test_shared_lengths(tq, P, B, G):
    """Rows that fill part of a tile, two tiles, and an odd tile; prefixes around the tile's edges."""
    run_shared(tq, B, G, 1, P, 33, 3, 3, 0, None, seed=P + B, q_size=0.5, od="bf16")


@pytest.mark.parametrize("page", [8, 16, 24, 72, 128, 256, 1000])
def test_shared_pages(tq, page):
    lens = [0, -1, 5, 130, 64, 1, -7, 129, 32]
    run_shared(tq, 9, 8, 2, 700, 130, 4, 2, page, lens, seed=page, od="bf16")
    run_shared(tq, 9, 8, 2, 391, 130, 2, 4, page, lens, seed=page, slack=300)


@pytest.mark.parametrize("B,Hq,Hkv,P,T", [(64, 28, 4, 5003, 100), (16, 32, 8, 20011, 300), (2, 8, 8, 9000, 2000),
                                          (200, 16, 2, 700, 20), (300, 64, 8, 200, 16)])
def test_shared_many(tq, B, Hq, Hkv, P, T):
    """More CTAs than SMs, many ranges of a prefix, own tokens that outnumber it."""
    lens = [(b * 37) % (T + 1) if b % 9 else -1 for b in range(B)]
    run_shared(tq, B, Hq, Hkv, P, T, 3, 3, 0, lens, seed=B + P, od="f16", q_size=2.0)


def test_shared_prefix_len(tq):
    """The prefix's length from the device: none, below, at and above its bound; one plan, one captured graph."""
    c = Case(6, 8, 2, 600, 50, 4, 3, 0, [50, 0, 10, -1, 1, 33], seed=3)
    c.prefix_len = i32([600])
    args, kw, out = c.args(tq, "f32")
    tq.tq_attn_decode_shared(*args, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_attn_decode_shared(*args, **kw)
    for n in (600, 0, 1, 128, 385, 599, 7777, -5):
        kw["prefix_len"].fill_(n)
        out.fill_(float("nan"))
        graph.replay()
        P = min(max(n, 0), 600)
        c.check(out, attend_reference(c.q.double().numpy(), c.kp[:, :P], c.vp[:, :P], c.ko, c.vo, c.eff, 4, 3))
    assert torch.all(out[1] == 0) and torch.all(out[3] == 0)   # no token at all; no sequence


@pytest.mark.parametrize("loud", [2e-4, 1e-2, 30.0, 1000.0, 3000.0])
def test_shared_norms_of_any_size(tq, loud):
    run_shared(tq, 33, 8, 1, 500, 20, 4, 4, 0, None, seed=5, loud=loud, q_size=min(1.0, 1 / loud))


def test_shared_loud_values_far_from_the_queries(tq):
    """A value of the largest norm under a key that no query looks at, value norms that grow along the prefix."""
    c = Case(20, 8, 1, 900, 8, 3, 3, 0, None, seed=6)
    norm = np.exp(np.linspace(-8, 9, 900))
    norm[5] = 60000.0
    h = codec.fp16_rne(norm)
    v = c.v_prefix.cpu().numpy()
    idx, old = codec.unpack_block(v[0, :900], 3)
    v[0, :900] = codec.pack_block(idx, h, 3)
    c.v_prefix = torch.from_numpy(v).cuda()
    c.vp = (c.vp[0] / codec.norm_value(old)[:, None] * codec.norm_value(h)[:, None])[None]
    args, kw, out = c.args(tq, "f32")
    tq.tq_attn_decode_shared(*args, **kw)
    c.check(out)


@pytest.mark.parametrize("B,P", [(3, 300), (40, 300), (40, 1000)])
@pytest.mark.parametrize("down", [False, True])
def test_shared_scores_that_grow(tq, B, P, down):
    """Key norms that grow (or shrink) along the prefix by four orders of magnitude: the references of the rows'
    exponents move in every tile, in its first and its second half."""
    c = Case(B, 8, 1, P, 8, 2, 3, 0, None, seed=7, q_size=0.5)
    norm = np.exp(np.linspace(-3, 7, P))[::-1 if down else 1]
    h = codec.fp16_rne(norm)
    k = c.k_prefix.cpu().numpy()
    idx, old = codec.unpack_block(k[0, :P], 2)
    k[0, :P] = codec.pack_block(idx, h, 2)
    c.k_prefix = torch.from_numpy(k).cuda()
    c.kp = (c.kp[0] / codec.norm_value(old)[:, None] * codec.norm_value(h)[:, None])[None]
    args, kw, out = c.args(tq, "f32")
    tq.tq_attn_decode_shared(*args, **kw)
    c.check(out)


def test_shared_equals_plain_decode(tq):
    """The same tokens as one cache of each sequence: within both calls' tolerances of each other."""
    c = Case(4, 8, 2, 320, 64, 4, 2, 64, [64, 0, 17, 40], seed=9)
    args, kw, out = c.args(tq, "f32")
    tq.tq_attn_decode_shared(*args, **kw)
    table = c.full.clone()[:, :6].contiguous()
    ref = torch.empty_like(out)
    ws = torch.empty(tq.tq_attn_workspace_bytes(4, 8, 2, 384), dtype=torch.uint8, device="cuda")
    tq.tq_attn_decode_paged(c.q.cuda(), c.k, args[4], c.v, args[6], table, 64, ref, 384, SCALE, args[12],
                            seq_lens=i32([384, 320, 337, 360]), workspace=ws)
    _, tol = c.check(out)
    # (there values are fp16 without a factor: 2^-12)
    _, tol2 = attend_reference(c.q.double().numpy(), c.kp, c.vp, c.ko, c.vo, c.eff, 4, 2, eps_v=2.0**-12)
    assert np.all(np.abs((out - ref).double().cpu().numpy()) <= tol + tol2)


def test_shared_not_finite(tq):
    """NaN and infinite keys reach the queries that see them: a prefix's, every sequence; an own token's, its own."""
    for P in (100, 300):
        c = Case(3, 4, 1, P, 20, 4, 2, 0, None, seed=11)
        args, kw, out = c.args(tq, "f32")
        clean = c.k_prefix.clone()
        for bits in (0x7E00, 0x7C00):                          # NaN, infinity
            c.k_prefix[0, 50, 0], c.k_prefix[0, 50, 1] = bits & 255, bits >> 8
            tq.tq_attn_decode_shared(*args, **kw)
            s = SCALE * c.q.double().numpy() @ (c.kp[0, 50] / np.abs(c.kp[0, 50]).max())
            if bits == 0x7E00:
                assert torch.isnan(out).all()
            else:                                              # +inf scores: NaN; -inf: the key has no weight
                bad = torch.isnan(out).all(-1).cpu().numpy()
                assert np.array_equal(bad, s > 0) and torch.isfinite(out.cpu()[~torch.from_numpy(bad)]).all()
            c.k_prefix.copy_(clean)
        k = c.k.clone()
        c.k[1, 0, 3, 0], c.k[1, 0, 3, 1] = 0x00, 0x7E
        tq.tq_attn_decode_shared(*args, **kw)
        assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()
        c.k.copy_(k)
        c.v_prefix[0, 2, 0], c.v_prefix[0, 2, 1] = 0x00, 0x7E   # a NaN value
        tq.tq_attn_decode_shared(*args, **kw)
        assert torch.isnan(out).all()
    assert tq.tq_device_status() == tq.TQ_OK


def test_shared_streams(tq):
    """Two streams at once with workspaces of their own; two captured graphs that share one, replayed in order."""
    cases = [Case(20, 16, 2, 2000, 100, 3, 3, 0, None, seed=20), Case(5, 8, 2, 900, 64, 4, 2, 16, None, seed=21)]
    calls = [c.args(tq, "bf16") for c in cases]
    want = []
    for a, kw, out in calls:
        tq.tq_attn_decode_shared(*a, **kw)
        want.append(out.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (a, kw, out) in zip(streams, calls):
            tq.tq_attn_decode_shared(*a, **kw, stream=s)
    torch.cuda.synchronize()
    for (a, kw, out), w in zip(calls, want):
        assert torch.equal(out, w)
    ws = max((a[8] for a, _, _ in calls), key=lambda t: t.numel())
    graphs = []
    for c in cases:
        a, kw, out = c.args(tq, "bf16", ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_attn_decode_shared(*a, **kw)
        graphs.append((g, out, a, kw))
    for _ in range(3):
        for g, out, _, _ in graphs:
            g.replay()
    for (g, out, _, _), w in zip(graphs, want):
        assert torch.equal(out, w)


def test_shared_wait_that_runs_out(tq):
    """With the copies' waits made to run out the call returns, the event is recorded, and the next call is right."""
    c = Case(30, 16, 2, 700, 40, 4, 4, 0, None, seed=30)
    args, kw, out = c.args(tq, "f32")
    tq.tq_device_status(clear=True)
    tq.tq_debug_drop_copies(True)
    try:
        tq.tq_attn_decode_shared(*args, **kw)
    finally:
        tq.tq_debug_drop_copies(False)
    assert tq.tq_device_status(clear=True) == tq.TQ_ERR_TIMEOUT
    assert not torch.isfinite(out).any()
    tq.tq_attn_decode_shared(*args, **kw)
    assert tq.tq_device_status() == tq.TQ_OK
    c.check(out)


# ---------------------------------------------------------------- all of them

def test_serving_loop(tq):
    """Prompts behind a shared prefix and decode steps after them: plan, norm and rotate, insert, attend, eagerly and
    as one captured graph, against the plain loop in 64 bits on the blocks that the loop wrote."""
    B, Hq, Hkv, page, P, kb, vb = 5, 8, 2, 16, 128, 4, 3
    hp, most, steps = P // page, 12, 6
    rng = np.random.default_rng(40)
    kcb, vcb = tq.tq_codebook_load(128, kb), tq.tq_codebook_load(128, vb)
    signs, rope = tq.tq_signs_from_seed(workloads.SIGN_SEED), tq.tq_rope_load(128, 1e6)
    sd = oracle.sign_diagonal(workloads.SIGN_SEED)
    books = oracle_books()
    pages = hp + B * 4 + 2
    kpool = torch.zeros(pages, Hkv, page, 66, dtype=torch.uint8, device="cuda")
    vpool = torch.zeros(pages, Hkv, page, 50, dtype=torch.uint8, device="cuda")
    wq, wk = (torch.from_numpy(1 + 0.2 * rng.standard_normal(128)).bfloat16().cuda() for _ in range(2))
    free, count = i32(rng.permutation(pages)), i32([pages])
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")

    def tokens(n):
        return torch.from_numpy(rng.standard_normal((n, Hq + 2 * Hkv, 128))).bfloat16().cuda()

    # the prefix: one request's prompt, whose pages head every row of the table
    held, lens = i32([0]), i32([0])
    seq, start = torch.empty_like(lens), torch.empty(2, dtype=torch.int32, device="cuda")
    dst, pos = torch.empty(P, dtype=torch.int64, device="cuda"), torch.empty(P, dtype=torch.int64, device="cuda")
    tq.tq_page_plan(lens, i32([P]), held, table[:1], free, count, page, Hkv, held, count, seq, start, dst, pos)
    x = tokens(P)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    tq.tq_norm_rope_apply(q, k, wq, wk, 1e-6, pos, rope, q, k)
    tq.tq_insert_kv(k, v, None, None, kcb, vcb, signs, kpool, vpool, dst, page)
    table[1:, :hp] = table[0, :hp]
    assert int(count) == pages - hp and int(seq) == P

    # a step of n tokens at most for the whole batch, the last of each request attending
    lens, held = i32([P] * B), i32([hp] * B)

    def state(n):
        return dict(x=tokens(n), fresh=i32([0] * B), seq=torch.empty_like(lens), start=i32([0] * (B + 1)),
                    dst=torch.empty(n, dtype=torch.int64, device="cuda"),
                    pos=torch.empty(n, dtype=torch.int64, device="cuda"), last=torch.zeros(B, dtype=torch.int64, device="cuda"),
                    q=torch.empty(n, Hq, 128, dtype=torch.bfloat16, device="cuda"),
                    out=torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda"),
                    ws=torch.empty(tq.tq_attn_shared_workspace_bytes(B, Hq, Hkv, P, (most - hp) * page),
                                   dtype=torch.uint8, device="cuda"))

    def step(s):
        tq.tq_page_plan(lens, s["fresh"], held, table, free, count, page, Hkv, held, count, s["seq"], s["start"],
                        s["dst"], s["pos"])
        k, v = s["x"][:, Hq:Hq + Hkv], s["x"][:, Hq + Hkv:]
        tq.tq_norm_rope_apply(s["x"][:, :Hq], k, wq, wk, 1e-6, s["pos"], rope, s["q"], k)
        tq.tq_insert_kv(k, v, None, None, kcb, vcb, signs, kpool, vpool, s["dst"], page)
        q = s["q"][s["last"]]
        tq.tq_attn_decode_shared(q, kpool, vpool, kpool, kcb, vpool, vcb, s["out"], s["ws"], P, (most - hp) * page, SCALE,
                                 signs, prefix_table=table[0, :hp], seq_lens=s["seq"] - P, block_table=table[:, hp:])
        lens.copy_(s["seq"])
        return q

    def check(s, q, fresh):
        L = lens.cpu().numpy()
        tb, kc, vc = table.cpu().numpy(), kpool.cpu().numpy(), vpool.cpu().numpy()
        own, pre = [], []
        for pool, bits in ((kc, kb), (vc, vb)):
            c = books[bits][0].astype(np.float32).astype(np.float64)
            vec = lambda blk: codec.decode(*codec.unpack_block(blk.reshape(-1, blk.shape[-1]), bits), c, sd).reshape(
                *blk.shape[:-1], 128)
            pre.append(vec(pool[tb[0, :hp]].transpose(1, 0, 2, 3).reshape(Hkv, P, -1)))
            rows = np.zeros((B, Hkv, (most - hp) * page, 128))
            for b in range(B):
                n = -(-(L[b] - P) // page)
                rows[b, :, :n * page] = 0 if n == 0 else vec(pool[tb[b, hp:hp + n]].transpose(1, 0, 2, 3).reshape(Hkv, n * page, -1))
            own.append(rows)
        want, tol = attend_reference(q.double().cpu().numpy(), pre[0], pre[1], own[0], own[1], L - P, kb, vb)
        eps = 2.0**-8
        err = np.abs(s["out"].double().cpu().numpy() - want)
        assert np.all(err <= tol * (1 + eps) + eps * np.abs(want) + 1e-37)

    fresh = [20, 3, 1, 0, 33]
    s = state(sum(fresh) + 3)
    s["fresh"].copy_(i32(fresh))
    s["last"].copy_(torch.tensor(np.maximum(np.cumsum(fresh) - 1, 0)))
    q = step(s)
    assert lens.tolist() == [P + n for n in fresh] and held.tolist() == [hp + -(-n // page) for n in fresh]
    check(s, q, fresh)

    d = state(B)
    d["fresh"].fill_(1)
    d["last"].copy_(torch.arange(B))
    check(d, step(d), [1] * B)
    x0, lens0, held0, count0 = d["x"].clone(), lens.clone(), held.clone(), count.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = step(d)
    assert torch.equal(lens, lens0) and torch.equal(held, held0) and torch.equal(count, count0)   # (captured, not run)
    for _ in range(steps):
        d["x"].copy_(tokens(B))
        graph.replay()
        check(d, q, [1] * B)
    assert lens.tolist() == [P + n + 1 + steps for n in fresh]
    rows = table.cpu().numpy()
    names = [rows[0, :hp].tolist()] + [rows[b, hp:int(held[b])].tolist() for b in range(B)]
    flat = sum(names, [])
    assert len(set(flat)) == len(flat) and int(count) == pages - len(flat)      # no page twice, none lost
    assert tq.tq_device_status() == tq.TQ_OK
