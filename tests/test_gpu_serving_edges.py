"""Rotary insert, weighted attention and eviction at the edges of what their
calls allow."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import oracle
from oracle import codec
from parity_util import oracle_books
from test_gpu_rope_insert import rotated
from turboquant_bit_kv_gb300 import workloads

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from turboquant_bit_kv_gb300 import tq as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("page", [40, 71582792, 100000008])
def test_attend_in_one_large_page(tq, page):
    """A page of any multiple of 8 tokens, far larger than the context too: the same bits as the contiguous cache."""
    T, bits = 109, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    cb, signs = tq.tq_codebook_load(128, bits), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    rows = torch.randn(2, T, 128, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 4, 128, generator=g, device="cuda")
    pages = -(-T // page)
    pools, flat = [], []
    for x in rows:
        pool = torch.empty(pages, 1, page, 34, dtype=torch.uint8, device="cuda")
        tq.tq_encode_kv(x, cb, signs, pool.view(-1, 34)[:T])
        pools.append(pool)
        flat.append(torch.zeros(1, 1, 112, 34, dtype=torch.uint8, device="cuda"))
        flat[-1][0, 0, :T] = pool.view(-1, 34)[:T]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(1, 4, 1, T), dtype=torch.uint8, device="cuda")
    got = []
    for (k, v), t in ((pools, table), (flat, None)):
        w, out = torch.zeros(1, 1, T, device="cuda"), torch.empty(1, 4, 128, device="cuda")
        tq.tq_attn_decode_weights(q, k, cb, v, cb, w, out, ws, T, SCALE, signs, block_table=t)
        got.append((w, out))
    assert torch.isfinite(got[0][1]).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---------------------------------------------------------------- decisions next to a boundary

def encoded_rows(x, bits, signs, zone=0.0):
    """Codes and norms of float64 rows by 64-bit arithmetic, the codes' coordinates shifted by zone; signs [128] of
    +-1."""
    norm = np.sqrt((x * x).sum(-1))
    y = (x * signs) @ oracle.hadamard(128).T / (np.sqrt(128) * norm[:, None]) + zone
    return np.searchsorted(oracle_books()[bits][2], y.astype(np.float32), side="right"), codec.fp16_rne(norm)


def check_rows(tq, x, pos, rope, bits, signs, rows, diagonal, keys=True):
    """Rows x [n, heads, 128] as keys (or as values), in one call and in calls of at most 24 tokens (large and small
    calls take different kernels), against rows [n * heads, 128] (float64, rotated).

    A coordinate nearer than 1e-11 to a boundary may fall either way: near a boundary the kernels decide in
    double-float, whose sines and cosines are off by less than 2^-38 together, sqrt(2) of it in a pair's sum, the
    norms of 64 pairs 8 of the row's at most: 8 sqrt(2) 2^-38 / sqrt(128) = 3.6e-12 of y.  Sums of 128 terms in
    double-float, the norm and its root add less than 40 * 2^-44."""
    n, heads = x.shape[:2]
    cb = tq.tq_codebook_load(128, bits)
    low, norm = encoded_rows(rows, bits, diagonal, -1e-11)
    high, _ = encoded_rows(rows, bits, diagonal, 1e-11)
    dst = torch.arange(n, device="cuda") * heads
    for step in (n, 24):
        cache = torch.zeros(n * heads, 2 + 16 * bits, dtype=torch.uint8, device="cuda")
        for i in range(0, n, step):
            p = None if rope is None else pos[:, i:i + step].contiguous()
            part, d = x[i:i + step], dst[i:i + step]
            if keys:
                tq.tq_insert_kv(part, None, p, rope, cb, None, signs, cache, None, d, 1)
            else:
                tq.tq_insert_kv(None, part, None, None, None, cb, signs, None, cache, d, 1)
        code, half = codec.unpack_block(cache.cpu().numpy(), bits)
        assert np.array_equal(half, norm)
        wrong = np.nonzero(((code < low) | (code > high)).any(-1))[0]
        assert wrong.size == 0, "%d of %d rows differ (calls of %d tokens), the first %s" % (
            wrong.size, n * heads, step, wrong[:5])


# angle (2^-32 turns) at which the float32 sine and cosine are off the furthest along the circle, 2.1 * 2^-24
WORST_ANGLE = 531149040


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("rot", [128, 96])
@pytest.mark.parametrize("bits", [2, 4])
def test_insert_of_rows_whose_errors_add_up(tq, style, rot, bits):
    """Keys whose pairs are all alike and turn by one angle: the errors of its sine and cosine add up over the row,
    in a coordinate that is within 2.5e-6 of a standard deviation of the boundary at 0."""
    n, heads, pairs = 3000, 5, rot // 2
    rope = tq.tq_rope_load(rot, style=style)
    tq.tq_rope_set_freqs(rope, [WORST_ANGLE * 2 * np.pi / 2**32] * pairs)
    rng = np.random.default_rng(rot + bits + style)
    pos = np.where(rng.random((1, n)) < 0.5, 1, -1)
    theta = pos[0, :, None, None] * (WORST_ANGLE * 2 * np.pi / 2**32)
    # rotated pairs (1, -1), each a little off; the rest of the row small
    ra, rb = (s + 1e-3 * rng.standard_normal((n, heads, pairs)) for s in (1.0, -1.0))
    rest = 1e-2 * rng.standard_normal((n, heads, 128 - rot))
    norm = np.sqrt((ra**2).sum(-1) + (rb**2).sum(-1) + (rest**2).sum(-1))
    target = rng.uniform(-2.5e-6, 2.5e-6, (n, heads)) * norm
    shift = (target - ra.sum(-1) - rb.sum(-1) - rest.sum(-1)) / rot
    ra, rb = ra + shift[..., None], rb + shift[..., None]
    a, b = ra * np.cos(theta) + rb * np.sin(theta), rb * np.cos(theta) - ra * np.sin(theta)
    x = np.zeros((n, heads, 128))
    i = np.arange(pairs)
    fi, se = (i, i + pairs) if style == 0 else (2 * i, 2 * i + 1)
    x[..., fi], x[..., se], x[..., rot:] = a, b, rest
    x = torch.from_numpy(x).float().cuda()
    turned = rotated(x.double().cpu().numpy(), pos, rope)[0].reshape(-1, 128)
    check_rows(tq, x, torch.from_numpy(pos).cuda(), rope, bits, tq.tq_signs(), turned, np.ones(128))


@pytest.mark.parametrize("keys", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_insert_of_rows_near_a_hadamard_row(tq, dtype, keys):
    """Rows of two magnitudes that cancel in one coordinate and agree in another: partial sums as large as sums of
    128 elements of the norm can be, and roundings that all go the same way."""
    n, heads, bits = 3000, 5, 4
    rng = np.random.default_rng(5)
    h, m = oracle.hadamard(128), n * heads
    j, k = rng.integers(1, 128, m), rng.integers(1, 128, m)
    same = h[j] == h[k]                                            # (half of the elements, or all)
    ulp = {"f32": 2.0**-23, "bf16": 2.0**-7, "f16": 2.0**-10}[dtype]
    hi = 1 + rng.integers(0, 64, (m, 1)) * ulp
    if dtype == "f32":
        hi = 1 + rng.integers(4, 2**22, (m, 1)) * ulp
    lo = hi + rng.integers(-3, 4, (m, 1)) * ulp
    diagonal = oracle.sign_diagonal(workloads.SIGN_SEED)
    x = diagonal * h[j] * np.where(same, hi, lo) * 2.0**rng.integers(-3, 4, (m, 1))
    few = rng.random((m, 128)) < 0.02
    x = np.where(few & (rng.random((m, 1)) < 0.5), x * 2.0**rng.integers(-22, 1, (m, 128)), x)
    x = torch.from_numpy(x.reshape(n, heads, 128)).to({"f32": torch.float32, "bf16": torch.bfloat16,
                                                       "f16": torch.float16}[dtype]).cuda()
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    rows = x.double().cpu().numpy().reshape(-1, 128)
    # sums of 128 values of 24 bits, 2^25 apart at most, are exact in 64 bits whatever their order
    check_rows(tq, x, None, None, bits, signs, rows, diagonal, keys)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("n", [20, 4000])
def test_insert_with_a_codebook_of_ones_own(tq, bits, n):
    """Boundaries moved off 0: a row of zeros takes the cell that 0 lies in, other rows theirs."""
    cb = tq.tq_codebook_load(128, bits)
    moved = np.array(cb.boundaries[:cb.levels - 1], np.float32) + np.float32(0.003)
    for i, b in enumerate(moved):
        cb.boundaries[i] = b
    heads = 5
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((n, heads, 128))
    x[::3] = 0
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cache = torch.zeros(n * heads, 2 + 16 * bits, dtype=torch.uint8, device="cuda")
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    tq.tq_insert_kv(x, None, None, None, cb, None, signs, cache, None, torch.arange(n, device="cuda") * heads, 1)
    idx, norm, _ = codec.encode(x.double().cpu().numpy().reshape(-1, 128), oracle.sign_diagonal(workloads.SIGN_SEED), moved)
    assert np.array_equal(cache.cpu().numpy(), codec.pack_block(idx, norm, bits))


@pytest.mark.parametrize("heads", [1, 2, 3, 9])
@pytest.mark.parametrize("kind", ["random", "boundary"])
def test_insert_of_many_rows_by_heads(tq, heads, kind):
    """Large calls by number of heads (one and two heads take several tiles of tokens at once): random rows, some of
    which are taken again, and rows that all are (more of them than a CTA can list)."""
    n, bits = 150000 // heads, 2
    g = torch.Generator(device="cuda").manual_seed(heads)
    if kind == "random":
        x = torch.randn(n, heads, 128, generator=g, device="cuda").to(torch.float16)
    else:   # two elements of 128: most coordinates are exactly 0
        x = torch.zeros(n, heads, 128, device="cuda", dtype=torch.float16)
        at = torch.randint(0, 127, (n, heads, 1), generator=g, device="cuda")
        x.scatter_(2, at, 1.0).scatter_(2, at + 1, 1.0)
    cb, signs = tq.tq_codebook_load(128, bits), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    cache = torch.full((n * heads, 34), 171, dtype=torch.uint8, device="cuda")
    dst = torch.arange(n, device="cuda") * heads
    dst[::7] = -1
    tq.tq_insert_kv(None, x, None, None, None, cb, signs, None, cache, dst, 1)
    rows = x.double().cpu().numpy().reshape(-1, 128)
    idx, norm, _ = codec.encode(rows, oracle.sign_diagonal(workloads.SIGN_SEED), oracle_books()[bits][2])
    want = codec.pack_block(idx, norm, bits).reshape(n, heads, 34)
    want[::7] = 171
    assert np.array_equal(cache.cpu().numpy().reshape(n, heads, 34), want)


def test_insert_of_very_many_tokens(tq):
    """A call of several launches gives what calls of its parts give."""
    n, bits = 13_000_000, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n // 100, 1, 128, generator=g, device="cuda").to(torch.bfloat16).repeat(100, 1, 1)
    pos = torch.randint(0, 10**6, (2, n), generator=g, device="cuda")
    rope = tq.tq_rope_load(128, sections=[30, 34])
    dst = torch.arange(n, device="cuda").flip(0).contiguous()
    cb, signs = tq.tq_codebook_load(128, bits), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    caches = [torch.full((n, 34), 171, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for cache, step in zip(caches, (n, 1_000_003)):
        for i in range(0, n, step):
            tq.tq_insert_kv(x[i:i + step], None, pos[:, i:i + step].contiguous(), rope, cb, None, signs, cache, None,
                            dst[i:i + step], 1)
    assert torch.equal(caches[0], caches[1])
    assert not (caches[0][:, 2:] == 171).all(1).any()


# ---------------------------------------------------------------- far positions

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("far", [2**32, 2**37, 2**40, 2**50, 2**53])
def test_apply_far_positions_follow_the_frequencies(tq, far):
    """Angles against position times frequency in 80 digits: a rope's turns are whole numbers of 2^-64, so an angle is
    off by 2 pi |position| 2^-64 at most, on top of sine and cosine (2^-22 of a pair of ones, as for near
    positions)."""
    getcontext().prec = 80
    freqs = [500000.0 ** (-2.0 * i / 128) for i in range(64)]
    rope = tq.tq_rope_set_freqs(tq.tq_rope_load(128), freqs)
    where = [far, -far, far - 1, -far + 12345, far // 3]
    x = torch.zeros(len(where), 1, 128, device="cuda")
    x[..., :64] = 1.0
    out = torch.empty_like(x)
    tq.tq_rope_apply(x, torch.tensor(where, device="cuda"), rope, out)
    angle = np.array([[float(Decimal(p) * Decimal(f) % (2 * PI)) for f in freqs] for p in where])
    tol = 2.0**-22 + 2 * np.pi * 2.0**-64 * abs(far) + 2.0**-50
    got = out[:, 0].double().cpu().numpy()
    assert np.abs(got[:, :64] - np.cos(angle)).max() <= tol
    assert np.abs(got[:, 64:] - np.sin(angle)).max() <= tol
