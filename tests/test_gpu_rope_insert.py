"""Rotary positions and quantise-on-insert of new tokens against plain
64-bit computations.

Angles: 2 pi times the pair's turn times the position modulo 2^64, the turn
as an integer (its own test compares it with the frequency).

Tolerances.  tq_rope_apply: sine and cosine are off by at most 2^-23 (the
Taylor remainders below 2^-29, the float32 angle, polynomial and its rounding
half an ulp each), the two products and the sum by half an ulp each, so an
element by at most 2^-22 (|a| + |b|), plus one rounding to the output type,
eps / 2 of the value.  tq_insert_kv: codes and norms equal to those of the
64-bit computation, without exception."""

import numpy as np
import pytest
import torch

import oracle
from oracle import codec
from parity_util import oracle_books
from turboquant_bit_kv_gb300 import workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from turboquant_bit_kv_gb300 import tq as mod
    mod.lib()
    return mod


def angles(rope, pos):
    """cos, sin [n, pairs] (float64) of positions [axes, n]."""
    n = rope.rot_dim // 2
    turn = np.array(rope.turn[:n], np.uint64)
    axis = np.array(rope.axis[:n])
    with np.errstate(over="ignore"):
        frac = pos.astype(np.uint64)[axis].T * turn
    t = frac.astype(np.int64).astype(np.float64) * (2 * np.pi / 2.0**64)
    return np.cos(t), np.sin(t)


def rotated(x, pos, rope):
    """x float64 [n, heads, 128] -> rotated, and |a| + |b| of each element's pair."""
    cos, sin = (v[:, None] for v in angles(rope, pos))
    n = rope.rot_dim // 2
    i = np.arange(n)
    fi, se = (i, i + n) if rope.style == 0 else (2 * i, 2 * i + 1)
    out, size = x.copy(), np.zeros_like(x)
    a, b = x[..., fi], x[..., se]
    out[..., fi], out[..., se] = a * cos - b * sin, b * cos + a * sin
    size[..., fi] = size[..., se] = np.abs(a) + np.abs(b)
    return out, size


ROPES = [dict(), dict(sections=[16, 24, 24], base=1e6), dict(sections=[24, 20, 20], interleaved=True),
         dict(style=1, sections=[30, 34]), dict(rot_dim=64), dict(rot_dim=96, sections=[10, 20, 18]),
         dict(rot_dim=32, style=1), dict(rot_dim=96, style=1, base=500.0), dict(rot_dim=32)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kw", ROPES)
@pytest.mark.parametrize("n,heads", [(1, 1), (7, 5), (130, 32), (3000, 3)])
def test_apply(tq, dtype, kw, n, heads):
    rope = tq.tq_rope_load(**kw)
    g = torch.Generator(device="cuda").manual_seed(n * 100 + heads)
    buf = torch.randn(n, heads + 3, 128, generator=g, device="cuda").to(DT[dtype])
    x = buf[:, 1:heads + 1]                                    # strided rows
    far = torch.randint(-2**40, 2**62, (rope.axes, n), generator=g, device="cuda")
    near = torch.randint(0, 200000, (rope.axes, n), generator=g, device="cuda")
    for pos in (near, far):
        out = torch.full((n, heads + 1, 128), 7.0, dtype=DT[dtype], device="cuda")
        before = buf.clone()
        tq.tq_rope_apply(x, pos, rope, out[:, :heads])
        assert torch.equal(buf, before) and torch.all(out[:, heads] == 7.0)
        want, size = rotated(x.double().cpu().numpy(), pos.cpu().numpy(), rope)
        err = np.abs(out[:, :heads].double().cpu().numpy() - want)
        eps = torch.finfo(DT[dtype]).eps / 2
        tiny = torch.finfo(DT[dtype]).smallest_normal * eps * 2
        assert np.all(err <= eps * np.abs(want) + 2.0**-22 * size * (1 + eps) + tiny)
        flat = out[..., rope.rot_dim:][:, :heads]
        assert torch.equal(flat, x[..., rope.rot_dim:])        # not rotated: copied
        tq.tq_rope_apply(x, pos, rope, x)                      # in place
        assert torch.equal(x, out[:, :heads])
        assert torch.equal(buf[:, 0], before[:, 0]) and torch.equal(buf[:, heads + 1:], before[:, heads + 1:])
        buf.copy_(before)


def test_apply_near_positions_follow_the_frequencies(tq):
    rope = tq.tq_rope_load(128, 1e6)
    pos = torch.tensor([0, 1, 4097, 131072, 1000000, -3], device="cuda")
    x = torch.zeros(6, 1, 128, device="cuda")
    x[..., :64] = 1.0
    out = torch.empty_like(x)
    tq.tq_rope_apply(x, pos, rope, out)
    t = pos.cpu().double()[:, None] * torch.tensor([1e6 ** (-2.0 * i / 128) for i in range(64)], dtype=torch.float64)
    # pos * f in double: off by 2^-53 of the angle (10^6: 1e-10)
    assert torch.allclose(out[:, 0, :64].double().cpu(), t.cos(), rtol=0, atol=2.0**-22)
    assert torch.allclose(out[:, 0, 64:].double().cpu(), t.sin(), rtol=0, atol=2.0**-22)


def test_apply_keeps_infinities_and_nan_in_their_pairs(tq):
    rope = tq.tq_rope_load(64)
    x = torch.ones(2, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[0, 0, 5], x[1, 1, 40], x[1, 0, 100] = float("inf"), float("nan"), float("inf")
    out = torch.empty_like(x)
    tq.tq_rope_apply(x, torch.tensor([3, 4], device="cuda"), rope, out)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 5] = want[0, 0, 37] = want[1, 1, 40] = want[1, 1, 8] = want[1, 0, 100] = True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------- insert

def encoded(x, bits):
    """Oracle blocks of float64 rows [n, 128]; rows with a non-finite element get codes 0."""
    s = oracle.sign_diagonal(workloads.SIGN_SEED)
    fine = np.isfinite(x).all(-1)
    idx, norm, _ = codec.encode(np.where(fine[:, None], x, 0.0), s, oracle_books()[bits][2])
    idx[~fine] = 0
    return codec.pack_block(idx, norm, bits), fine


def check_side(tq, cache, x, bits, dst, hs, before):
    """The cache against the oracle; untouched blocks as before."""
    got, want = cache.cpu().numpy(), before.cpu().numpy().copy()
    blocks, fine = encoded(x.reshape(-1, 128), bits)
    n, heads = x.shape[:2]
    at = dst[:, None] + np.arange(heads) * hs
    ok = ((at >= 0) & (dst[:, None] >= 0) & (at < len(want))).reshape(-1)
    want[at.reshape(-1)[ok]] = blocks[ok]
    odd = at.reshape(-1)[ok & ~fine]
    norms = got[odd][:, :2].copy().view(np.float16)
    assert not np.isfinite(norms).any()
    got[odd, :2] = want[odd, :2]
    wrong = np.nonzero((got != want).any(-1))[0]
    assert wrong.size == 0, (wrong[:5], got[wrong[:1]], want[wrong[:1]])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 2), (3, 3), (2, 4)])
@pytest.mark.parametrize("kw", [None] + ROPES)
def test_insert_is_exact(tq, dtype, kb, vb, kw):
    n, heads, T_cap = 533, 5, 600
    rope = None if kw is None else tq.tq_rope_load(**kw)
    g = torch.Generator(device="cuda").manual_seed(kb * 10 + vb)
    loud = torch.exp(torch.randn(2 * heads, 128, generator=g, device="cuda"))
    kv = (torch.randn(n, 2 * heads, 128, generator=g, device="cuda") * loud).to(DT[dtype])
    kv[7] = 0
    kv[8, 0, 3] = float("inf")
    kv[9, 6, 100] = float("nan")
    kv[10] *= 2.0**-14 if dtype == "f16" else 2.0**-60
    kv[11, :, 1:] = 0                                          # one element carries the row
    if dtype != "f16":
        kv[12] *= 2.0**-70                                     # squares underflow in float32
        kv[13] *= 2.0**90                                      # and overflow
    k, v = kv[:, :heads], kv[:, heads:]
    pos = torch.randint(0, 1000000, (3, n), generator=g, device="cuda")[:1 if rope is None else rope.axes].contiguous()
    dst = torch.randperm(T_cap, generator=g, device="cuda")[:n]
    dst[::9] = -1
    dst[5] = 10**9                                             # past the cache: not written
    sizes = 2 + 16 * kb, 2 + 16 * vb
    caches = [torch.randint(0, 256, (heads * T_cap, z), generator=g, device="cuda", dtype=torch.uint8) for z in sizes]
    before = [c.clone() for c in caches]
    books = tq.tq_codebook_load(128, kb), tq.tq_codebook_load(128, vb)
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    tq.tq_insert_kv(k, v, pos, rope, books[0], books[1], signs, caches[0], caches[1], dst, T_cap)
    kx = k.double().cpu().numpy()
    if rope is not None:
        with np.errstate(invalid="ignore"):
            kx = rotated(kx, pos.cpu().numpy(), rope)[0]
    d = dst.cpu().numpy()
    check_side(tq, caches[0], kx, kb, d, T_cap, before[0])
    check_side(tq, caches[1], v.double().cpu().numpy(), vb, d, T_cap, before[1])


def test_insert_many_rows_is_exact(tq):
    """640 thousand rows: some hundred coordinates lie within float32 noise of a boundary."""
    n, heads = 20000, 32
    rope = tq.tq_rope_load(128, 1e6, sections=[16, 24, 24])
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(n, heads, 128, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 130000, (3, n), generator=g, device="cuda")
    cache = torch.zeros(heads * n, 66, dtype=torch.uint8, device="cuda")
    cb, signs = tq.tq_codebook_load(128, 4), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    tq.tq_insert_kv(k, None, pos, rope, cb, None, signs, cache, None, torch.arange(n, device="cuda"), n)
    cos, sin = (torch.from_numpy(v).cuda()[:, None] for v in angles(rope, pos.cpu().numpy()))
    h = torch.from_numpy(oracle.hadamard(128) * oracle.sign_diagonal(workloads.SIGN_SEED) / np.sqrt(128)).cuda()
    bounds = torch.from_numpy(oracle_books()[4][2]).cuda()
    for i in range(0, n, 4000):
        x = k[i:i + 4000].double()
        a, b = x[..., :64], x[..., 64:]
        c, s = cos[i:i + 4000], sin[i:i + 4000]
        x = torch.cat([a * c - b * s, b * c + a * s], -1)
        norm = x.norm(dim=-1)
        code = torch.bucketize(((x @ h.T) / norm[..., None]).float(), bounds, right=True)
        got = cache.view(heads, n, 66)[:, i:i + 4000].transpose(0, 1)
        # (numpy rounds float64 to fp16 once; torch's conversion goes through float32)
        half = codec.fp16_rne(norm.cpu().numpy()).view(np.int16)
        assert np.array_equal(got[..., :2].contiguous().view(torch.int16)[..., 0].cpu().numpy(), half)
        assert torch.equal(got[..., 2:], (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8))


@pytest.mark.parametrize("n,heads,page", [(1, 1, 8), (16, 8, 16), (33, 4, 5), (100, 9, 64)])
def test_insert_into_pages(tq, n, heads, page):
    pages = -(-n // page) + 2
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, 2 * heads, 128, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    dst = table[t // page] * heads * page + t % page
    cb, signs = tq.tq_codebook_load(128, 3), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    pools = [torch.full((pages, heads, page, 50), 171, dtype=torch.uint8, device="cuda") for _ in range(2)]
    before = [p.clone().view(-1, 50) for p in pools]
    tq.tq_insert_kv(x[:, :heads], x[:, heads:], None, None, cb, cb, signs, pools[0], pools[1], dst, page)
    for pool, rows, b in zip(pools, (x[:, :heads], x[:, heads:]), before):
        check_side(tq, pool.view(-1, 50), rows.double().cpu().numpy(), 3, dst.cpu().numpy(), page, b)
    only = [torch.full((pages, heads, page, 50), 171, dtype=torch.uint8, device="cuda") for _ in range(2)]
    tq.tq_insert_kv(x[:, :heads], None, None, None, cb, None, signs, only[0], None, dst, page)
    tq.tq_insert_kv(None, x[:, heads:], None, None, None, cb, signs, None, only[1], dst, page)
    assert torch.equal(only[0], pools[0]) and torch.equal(only[1], pools[1])


def test_insert_consecutive_slots_at_every_offset(tq):
    """Runs of 16 slots leave as one piece where they start at a 16-byte boundary, else block by block."""
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    x = torch.randn(64, 2, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    for bits in (2, 3, 4):
        cb = tq.tq_codebook_load(128, bits)
        for off in range(9):
            cache = torch.zeros(2 * 80, 2 + 16 * bits, dtype=torch.uint8, device="cuda")
            before = cache.clone()
            dst = torch.arange(64, device="cuda") + off
            tq.tq_insert_kv(x, None, None, None, cb, None, signs, cache, None, dst, 80)
            check_side(tq, cache, x.double().cpu().numpy(), bits, dst.cpu().numpy(), 80, before)


def inserted(tq, k, v, pos, rope, bits, dst, heads, T_cap, cuts):
    """Caches (filled with 171) after inserting the tokens in calls cut at cuts."""
    caches = [torch.full((heads * T_cap, 2 + 16 * b), 171, dtype=torch.uint8, device="cuda") for b in bits]
    books = [tq.tq_codebook_load(128, b) for b in bits]
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    for i, j in zip(cuts, cuts[1:]):
        p = None if rope is None else pos[:, i:j].contiguous()
        tq.tq_insert_kv(None if k is None else k[i:j], None if v is None else v[i:j], p, rope, books[0], books[1], signs,
                        None if k is None else caches[0], None if v is None else caches[1], dst[i:j], T_cap)
    return caches


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(1 + len(ROPES)))
def test_insert_of_many_tokens_equals_inserts_of_few(tq, dtype, case):
    """A call's blocks do not depend on its size (large and small calls take
    different kernels), whatever the rows hold."""
    n, heads, T_cap = 8209, 5, 8300
    bits = [(4, 2), (3, 3), (2, 4)][case % 3]
    rope = None if case == 0 else tq.tq_rope_load(**ROPES[case - 1])
    g = torch.Generator(device="cuda").manual_seed(case)
    loud = torch.exp(torch.randn(2 * heads, 128, generator=g, device="cuda"))
    kv = (torch.randn(n, 2 * heads, 128, generator=g, device="cuda") * loud).to(DT[dtype])
    kv[7::500] = 0
    kv[8::500, 0, 3] = float("inf")
    kv[9::500, 6, 100] = float("nan")
    kv[10::500] *= 2.0**-14 if dtype == "f16" else 2.0**-60
    kv[11::500, :, 1:] = 0
    kv[14::500] = torch.randint(-3, 4, kv[14::500].shape, generator=g, device="cuda").to(DT[dtype])
    if dtype != "f16":
        kv[12::500] *= 2.0**-70
        kv[13::500] *= 2.0**90
    pos = torch.randint(-10**6, 10**6, (3, n), generator=g, device="cuda")[:1 if rope is None else rope.axes].contiguous()
    dst = torch.randperm(T_cap, generator=g, device="cuda")[:n]
    dst[::9] = -1
    dst[5] = 10**9
    k, v = kv[:, :heads], kv[:, heads:]
    cuts = [0, 1, 3, 19, 36, 500, 1000, 2001, 4000, 6000, 8000, n]
    one = inserted(tq, k, v, pos, rope, bits, dst, heads, T_cap, [0, n])
    for a, b in zip(one, inserted(tq, k, v, pos, rope, bits, dst, heads, T_cap, cuts)):
        assert torch.equal(a, b)
    assert torch.equal(one[0], inserted(tq, k, None, pos, rope, bits, dst, heads, T_cap, [0, n])[0])
    assert torch.equal(one[1], inserted(tq, None, v, pos, rope, bits, dst, heads, T_cap, cuts)[1])


@pytest.mark.parametrize("n", [40, 6000])
@pytest.mark.parametrize("dtype,bits,ones", [("bf16", 4, 128), ("f16", 3, 6), ("f32", 2, 2), ("bf16", 2, 32)])
def test_insert_of_coordinates_on_a_boundary(tq, n, dtype, bits, ones):
    """Rows of a few small integers: many coordinates are exactly 0, a
    boundary of every codebook (64-bit sums of integers are exact)."""
    heads = 5
    g = torch.Generator(device="cuda").manual_seed(ones)
    x = torch.zeros(n, heads, 128, device="cuda")
    x[..., :ones] = torch.randint(-2, 3, (n, heads, ones), generator=g, device="cuda").float()
    x = x.gather(2, torch.argsort(torch.rand(n, heads, 128, generator=g, device="cuda"), -1))
    dst = torch.arange(n, device="cuda")
    cache = inserted(tq, x.to(DT[dtype]), None, None, None, (bits, bits), dst, heads, n, [0, n])[0]
    before = torch.full_like(cache, 171)
    check_side(tq, cache, x.double().cpu().numpy(), bits, dst.cpu().numpy(), n, before)
