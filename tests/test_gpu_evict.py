"""Decode attention with accumulated weights, selection and compaction
against plain 64-bit computations, and a decode loop of all of them.

Tolerances of the attention.  With S = sum_t p_t ||v_t|| of a query head:
scores are products of operands split in two fp16 parts, off by 2^-21
relative and 2^-25 absolute per element, accumulated in float32 over 32
steps: ds = scale ||q|| n ||c|| (2^-21 + 32 * 2^-23) + n (|c|_1 + |Rq|_1
scale) 2^-25; a weight is off by 2 ds + 2^-17 of itself (the exponential and
sums of up to a few hundred partial terms in float32), its accumulator by
another 2^-23.  Outputs: that on every p, and value centroids rounded to fp16
(2^-12 of each value at worst): (2 ds + 2^-17 + 2^-12) S, plus the output
type's rounding, eps / 2 of the value."""

import numpy as np
import pytest
import torch

import oracle
from oracle import codec
from parity_util import oracle_books
from turboquant_bit_kv_gb300 import workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from turboquant_bit_kv_gb300 import tq as mod
    mod.lib()
    return mod


def cache_of(shape, bits, rng, loud=1.0):
    """Random blocks [*shape, bytes] and the vectors they stand for (float64)."""
    n = int(np.prod(shape))
    c, _, b32 = oracle_books()[bits]
    idx = np.searchsorted(b32 * np.sqrt(128), rng.standard_normal((n, 128)).astype(np.float32)).astype(np.uint8)
    norm = codec.fp16_rne(np.sqrt(128) * np.exp(0.3 * rng.standard_normal(n)) * loud)
    vec = codec.decode(idx, norm, c.astype(np.float32).astype(np.float64), oracle.sign_diagonal(workloads.SIGN_SEED))
    return codec.pack_block(idx, norm, bits).reshape(*shape, -1), vec.reshape(*shape, 128)


def reference(q, kv, vv, lens, w, decay):
    """out, weights and their tolerances (without the output type's rounding)."""
    B, Hq, _ = q.shape
    Hkv = kv.shape[1]
    G = Hq // Hkv
    out, tol_o = np.zeros((B, Hq, 128)), np.zeros((B, Hq, 1))
    new, tol_w = w.astype(np.float64).copy(), np.zeros(w.shape)
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        for h in range(Hkv):
            tot, tol = np.zeros(L), np.zeros(L)
            for g in range(G):
                x = q[b, h * G + g]
                s = SCALE * kv[b, h, :L] @ x
                n = np.linalg.norm(kv[b, h, :L], axis=-1).max()
                ds = SCALE * np.linalg.norm(x) * n * (2.0**-21 + 2.0**-18) + \
                    n * (12.0 + 12.0 * SCALE * np.linalg.norm(x)) * 2.0**-25
                p = np.exp(s - s.max())
                p /= p.sum()
                rel = 2 * ds + 2.0**-17
                out[b, h * G + g] = p @ vv[b, h, :L]
                tol_o[b, h * G + g] = (rel + 2.0**-12) * (p @ np.linalg.norm(vv[b, h, :L], axis=-1))
                tot += p
                tol += p * rel
            new[b, h, :L] = tot + (decay * new[b, h, :L] if decay else 0.0)
            tol_w[b, h, :L] = tol + 2.0**-23 * np.abs(new[b, h, :L])
    return out, tol_o, new, tol_w


def run_attend(tq, B, Hq, Hkv, T, kb, vb, page, lens, decay, qd, od, seed):
    rng = np.random.default_rng(seed)
    kblk, kv = cache_of((B, Hkv, T), kb, rng)
    vblk, vv = cache_of((B, Hkv, T), vb, rng)
    q = (torch.from_numpy(rng.standard_normal((B, Hq, 128))) * 2).to(DT[qd])
    w0 = np.abs(rng.standard_normal((B, Hkv, T + 5))).astype(np.float32)
    if decay == 0.0:
        w0[..., 1] = np.nan                       # overwritten, not multiplied
    w = torch.from_numpy(w0).cuda()
    table = None
    if page:
        pages = -(-T // page)
        ids = rng.permutation(B * pages + 3)[:B * pages].reshape(B, pages)
        table = torch.full((B, pages + 2), -1, dtype=torch.int32)      # entries past the context are not read
        table[:, :pages] = torch.from_numpy(ids)
        table = table.cuda()
        caches = []
        for blk in (kblk, vblk):
            pool = rng.integers(0, 256, (B * pages + 3, Hkv, page, blk.shape[-1]), dtype=np.uint8)
            for b in range(B):
                for i in range(pages):
                    part = blk[b, :, i * page:(i + 1) * page]
                    pool[ids[b, i], :, :part.shape[1]] = part
            caches.append(torch.from_numpy(pool).cuda())
    else:
        T_cap = (T + 7) // 8 * 8 + 8
        caches = []
        for blk in (kblk, vblk):
            full = rng.integers(0, 256, (B, Hkv, T_cap, blk.shape[-1]), dtype=np.uint8)
            full[:, :, :T] = blk
            caches.append(torch.from_numpy(full).cuda())
    seq = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    eff = [T] * B if lens is None else [min(max(n, 0), T) for n in lens]
    out = torch.full((B, Hq, 128), float("nan"), dtype=DT[od], device="cuda")
    ws = torch.full((tq.tq_attn_weights_workspace_bytes(B, Hq, Hkv, T),), 255, dtype=torch.uint8, device="cuda")
    args = (q.cuda(), caches[0], tq.tq_codebook_load(128, kb), caches[1], tq.tq_codebook_load(128, vb))
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    tq.tq_attn_decode_weights(*args, w, out, ws, T, SCALE, signs, seq_lens=seq, block_table=table, decay=decay)
    ref, tol_o, new, tol_w = reference(q.double().numpy(), kv, vv, eff, w0[..., :T], decay)
    eps = torch.finfo(DT[od]).eps / 2
    over = np.abs(out.double().cpu().numpy() - ref) / (tol_o * (1 + eps) + eps * np.abs(ref) + 1e-37)
    worst = np.unravel_index(np.nanargmax(over), over.shape)
    assert np.nanmax(over) <= 1 and np.isfinite(over).all(), (over.max(), worst, float(out[worst]), ref[worst])
    got = w.double().cpu().numpy()
    live = np.arange(T) < np.array(eff)[:, None]
    live = np.broadcast_to(live[:, None], (B, Hkv, T))
    assert np.all(np.abs(got[..., :T] - new)[live] <= tol_w[live] + 1e-37)
    assert np.array_equal(w.cpu().numpy()[..., :T][~live], w0[..., :T][~live], equal_nan=True)   # left as they were
    assert np.array_equal(w.cpu().numpy()[..., T:], w0[..., T:], equal_nan=True)
    # the same call again on the same accumulators' start gives the same bits
    w2, out2 = torch.from_numpy(w0).cuda(), torch.empty_like(out)
    tq.tq_attn_decode_weights(*args, w2, out2, ws, T, SCALE, signs, seq_lens=seq, block_table=table, decay=decay)
    assert torch.equal(w2.nan_to_num(7.0), w.nan_to_num(7.0)) and torch.equal(out2, out)


@pytest.mark.parametrize("kb", [2, 3, 4])
@pytest.mark.parametrize("vb", [2, 3, 4])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_attend_formats(tq, kb, vb, G):
    run_attend(tq, 3, 2 * G, 2, 203, kb, vb, 0, [203, 77, 0], 0.9, "bf16", "f32", kb * 100 + vb * 10 + G)
    run_attend(tq, 3, 2 * G, 2, 203, kb, vb, 64, [33, 203, -4], 1.0, "f16", "f16", kb * 100 + vb * 10 + G + 1)


@pytest.mark.parametrize("G", [2, 3, 5, 6, 8])
def test_attend_group_sizes(tq, G):
    run_attend(tq, 2, 3 * G, 3, 130, 4, 2, 32, [130, 129], 1.0, "f32", "bf16", G)


@pytest.mark.parametrize("T,B,Hkv,page", [(1, 1, 1, 0), (1, 3, 2, 32), (31, 2, 1, 0), (32, 1, 2, 32), (33, 1, 1, 64),
                                          (1025, 2, 2, 0), (2500, 1, 8, 96), (9001, 1, 1, 0)])
def test_attend_lengths(tq, T, B, Hkv, page):
    run_attend(tq, B, 4 * Hkv, Hkv, T, 4, 2, page, None, 1.0, "bf16", "bf16", T)
    run_attend(tq, B, 4 * Hkv, Hkv, T, 3, 3, page, [T + 100] + [T // 2] * (B - 1), 0.0, "bf16", "f32", T + 1)


@pytest.mark.parametrize("page", [8, 16, 24, 40, 48, 72, 96])
@pytest.mark.parametrize("kb,vb,G", [(4, 2, 4), (3, 3, 7), (2, 4, 1)])
def test_attend_page_sizes(tq, page, kb, vb, G):
    """Pages that end inside a chunk of 32 tokens; lengths at, before and after the ends of pages and chunks."""
    lens = [page, 8 * page, page - 1, page + 1, 333, 32, 31, 0]
    run_attend(tq, 8, 2 * G, 2, 8 * page + 5, kb, vb, page, lens, 0.5, "bf16", "f32", page + kb)


@pytest.mark.parametrize("B,Hkv,page", [(33, 2, 0), (70, 1, 32), (128, 1, 0)])
def test_attend_many_sequences(tq, B, Hkv, page):
    """Batches over 32 sequences, most of them short or empty, one long: the work is split over live chunks."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(-1, 70, B)]
    lens[B // 2] = 700
    lens[-1] = 1
    run_attend(tq, B, 2 * Hkv, Hkv, 700, 4, 2, page, lens, 1.0, "bf16", "f32", B)
    run_attend(tq, B, 5 * Hkv, Hkv, 200, 2, 3, page, [0] * (B - 1) + [7], 1.0, "bf16", "f32", B + 1)
    run_attend(tq, B, Hkv, Hkv, 40, 3, 4, page, [0] * B, 0.5, "f16", "bf16", B + 2)


def test_attend_matches_the_plain_decode(tq):
    """Same scores and values as tq_attn_decode: outputs agree to its tolerance, and the weights of a fresh
    accumulator add up to the group's heads."""
    B, Hq, Hkv, T = 2, 28, 4, 5000
    rng = np.random.default_rng(3)
    kb, vb = (torch.from_numpy(cache_of((B, Hkv, T), 3, rng)[0]).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((B, Hq, 128))).to(torch.bfloat16).cuda()
    cb, signs = tq.tq_codebook_load(128, 3), tq.tq_signs_from_seed(workloads.SIGN_SEED)
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(B, Hq, Hkv, T), dtype=torch.uint8, device="cuda")
    w = torch.zeros(B, Hkv, T, device="cuda")
    out, plain = (torch.empty(B, Hq, 128, device="cuda") for _ in range(2))
    tq.tq_attn_decode_weights(q, kb, cb, vb, cb, w, out, ws, T, SCALE, signs)
    tq.tq_attn_decode(q, kb, cb, vb, cb, plain, ws, T, SCALE, signs)
    assert ((out - plain).abs().amax(-1) <= 2e-3 * plain.abs().amax(-1)).all()
    # sums of 5000 float32 weights, each off by 2^-16 at most (scores up to 8)
    assert (w.double().sum(-1) - Hq // Hkv).abs().max() <= (Hq // Hkv) * 2.0**-15


def test_attend_extreme_queries(tq):
    """One key far ahead of the others: its weight is 1 and the rest underflow to 0; a NaN query spoils its own
    group and no other."""
    rng = np.random.default_rng(9)
    kblk, kv = cache_of((1, 2, 300), 4, rng)
    vblk, vv = cache_of((1, 2, 300), 2, rng)
    q = torch.zeros(1, 4, 128)
    q[0, 0] = torch.from_numpy(kv[0, 0, 17]) * 40
    q[0, 1] = -q[0, 0]
    q[0, 2] = float("nan")
    cbk, cbv = tq.tq_codebook_load(128, 4), tq.tq_codebook_load(128, 2)
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    caches = []
    for blk in (kblk, vblk):
        full = np.zeros((1, 2, 304, blk.shape[-1]), np.uint8)
        full[:, :, :300] = blk
        caches.append(torch.from_numpy(full).cuda())
    w, out = torch.zeros(1, 2, 300, device="cuda"), torch.empty(1, 4, 128, device="cuda")
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(1, 4, 2, 300), dtype=torch.uint8, device="cuda")
    tq.tq_attn_decode_weights(q.cuda(), caches[0], cbk, caches[1], cbv, w, out, ws, 300, SCALE, signs)
    assert torch.isfinite(out[0, :2]).all() and torch.isnan(out[0, 2]).all() and torch.isfinite(out[0, 3]).all()
    s = SCALE * kv[0, 0] @ q[0, :2].double().numpy().T
    p = np.exp(s - s.max(0))
    p = (p / p.sum(0)).sum(1)
    # scores up to 5000: off by 2^-18 of them at most
    assert np.abs(w[0, 0].double().cpu().numpy() - p).max() <= 2 * np.abs(s).max() * 2.0**-18
    assert torch.isnan(w[0, 1]).all()


@pytest.mark.parametrize("kb,vb,G", [(4, 2, 4), (3, 3, 7), (4, 4, 1), (2, 4, 8)])
def test_blocks_behind_the_sequence_do_not_matter(tq, kb, vb, G):
    """Stale blocks behind a sequence's last token, their norms NaN and infinite, change no bit."""
    B, Hkv, T = 2, 2, 96
    rng = np.random.default_rng(kb * vb)
    clean = [torch.from_numpy(cache_of((B, Hkv, T), n, rng)[0]).cuda() for n in (kb, vb)]
    q = torch.from_numpy(rng.standard_normal((B, Hkv * G, 128))).float().cuda()
    books, signs = [tq.tq_codebook_load(128, n) for n in (kb, vb)], tq.tq_signs_from_seed(workloads.SIGN_SEED)
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(B, Hkv * G, Hkv, T), dtype=torch.uint8, device="cuda")
    for L in (1, 31, 33, 45, 90):
        lens = torch.tensor([L, L + 3], dtype=torch.int32, device="cuda")
        got = []
        for bad in (False, True):
            kc, vc = (c.clone() for c in clean)
            if bad:
                for b in range(B):
                    for c in (kc, vc):
                        c[b, :, L + 3 * b:, :2] = torch.tensor([0, 0x7E], dtype=torch.uint8)      # NaN
                        c[b, 1, L + 3 * b::2, :2] = torch.tensor([0, 0x7C], dtype=torch.uint8)    # inf
            out, plain = (torch.empty(B, Hkv * G, 128, device="cuda") for _ in range(2))
            w = torch.zeros(B, Hkv, T, device="cuda")
            tq.tq_attn_decode_weights(q, kc, books[0], vc, books[1], w, out, ws, T, SCALE, signs, seq_lens=lens)
            tq.tq_attn_decode(q, kc, books[0], vc, books[1], plain, ws, T, SCALE, signs, seq_lens=lens)
            got.append((out, w, plain))
        assert all(torch.isfinite(x).all() for x in got[1])
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_attend_reports_a_wait_that_runs_out(tq):
    """Copies that never land (the test hook): the call returns, the status says so, outputs and weights are marked,
    and the next call is right again."""
    rng = np.random.default_rng(2)
    caches = [torch.from_numpy(cache_of((1, 2, 640), n, rng)[0]).cuda() for n in (4, 2)]
    q = torch.from_numpy(rng.standard_normal((1, 8, 128))).float().cuda()
    books, signs = [tq.tq_codebook_load(128, n) for n in (4, 2)], tq.tq_signs_from_seed(workloads.SIGN_SEED)
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(1, 8, 2, 640), dtype=torch.uint8, device="cuda")

    def call():
        w, out = torch.zeros(1, 2, 640, device="cuda"), torch.zeros(1, 8, 128, device="cuda")
        tq.tq_attn_decode_weights(q, caches[0], books[0], caches[1], books[1], w, out, ws, 640, SCALE, signs)
        return w, out

    tq.tq_device_status(clear=True)
    w0, out0 = call()
    assert tq.tq_device_status() == tq.TQ_OK
    tq.tq_debug_drop_copies(True)
    try:
        w1, out1 = call()
    finally:
        tq.tq_debug_drop_copies(False)
    assert tq.tq_device_status(clear=True) == tq.TQ_ERR_TIMEOUT
    assert not torch.isfinite(out1).all() and not torch.isfinite(w1).all()
    w2, out2 = call()
    assert tq.tq_device_status() == tq.TQ_OK
    assert torch.equal(w0, w2) and torch.equal(out0, out2)


# ---------------------------------------------------------------- selection

def select_reference(w, lens, keep, first, last):
    B, H, T = w.shape
    kept, new = np.full((B, H, keep), -1, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        L = T if lens is None else min(max(int(lens[b]), 0), T)
        new[b] = min(L, keep)
        for h in range(H):
            if L <= keep:
                kept[b, h, :L] = np.arange(L)
                continue
            mid = np.arange(first, L - last)
            x = w[b, h, mid].astype(np.float64)
            rank = np.where(np.isnan(x), np.inf, x)
            order = np.lexsort((mid, -rank, ~np.isnan(x)))
            top = mid[order[:keep - first - last]]
            kept[b, h] = np.sort(np.concatenate([np.arange(first), top, np.arange(L - last, L)]))
    return kept, new


@pytest.mark.parametrize("T,B,H,keep,first,last", [
    (1, 1, 1, 1, 0, 0), (2, 1, 1, 1, 0, 0), (2, 2, 1, 1, 0, 1), (33, 3, 2, 7, 2, 3), (1000, 2, 3, 500, 4, 100),
    (4096, 1, 8, 1024, 4, 256), (5000, 2, 2, 4999, 0, 0), (5000, 2, 2, 10, 4, 6), (5000, 1, 1, 8000, 1, 1),
    (32769, 3, 2, 16384, 4, 1000), (70001, 1, 2, 20000, 0, 0), (400003, 1, 1, 100000, 4, 64)])
@pytest.mark.parametrize("kind", ["smooth", "ties", "odd"])
def test_select(tq, T, B, H, keep, first, last, kind):
    rng = np.random.default_rng(T + keep)
    w = np.exp(2 * rng.standard_normal((B, H, T))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w)
        w[0] = 1.0
    if kind == "odd":
        odd = np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -1.0, 1.0], np.float32)
        w = odd[rng.integers(0, len(odd), (B, H, T))]
    lens = None if kind == "smooth" else [T] + [max(1, T * 2 // 3), -1][:B - 1]
    wide = torch.full((B, H, T + 3), float("nan"), device="cuda")
    wide[..., :T] = torch.from_numpy(w)
    kept = torch.full((B, H, keep), -7, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    seq = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    tq.tq_evict_select(wide, kept, new, T, first, last, seq_lens=seq)
    want, want_new = select_reference(w, lens, keep, first, last)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), want_new)


# ---------------------------------------------------------------- compaction

def compact_reference(blk, kept, new):
    out = blk.copy()
    for b in range(kept.shape[0]):
        for h in range(kept.shape[1]):
            src = kept[b, h, :new[b]]
            out[b, h, :new[b]] = blk[b, h, src]
    return out


@pytest.mark.parametrize("T,B,H,keep,page", [(1, 1, 1, 1, 0), (40, 2, 3, 9, 0), (40, 2, 3, 9, 7), (1000, 3, 2, 500, 16),
                                             (4096, 1, 8, 1024, 0), (4099, 2, 4, 4000, 64), (3000, 40, 8, 1500, 0)])
@pytest.mark.parametrize("kbytes,vbytes", [(66, 34), (50, 130), (2, 0), (512, 66)])
def test_compact(tq, T, B, H, keep, page, kbytes, vbytes):
    if kbytes == 512 and B == 40:
        kbytes = 34
    rng = np.random.default_rng(T + kbytes)
    lens = np.array([T] + [max(keep // 2, 1), T - T // 4][:B - 1] + [T] * max(0, B - 3))
    w = rng.random((B, H, T)).astype(np.float32)
    kept, new = select_reference(w, lens, keep, min(2, keep), 0)
    cap = -(-T // page) * page if page else T + 3
    logical = [rng.integers(0, 256, (B, H, cap, z), dtype=np.uint8) for z in (kbytes, vbytes) if z]
    table = None
    if page:
        pages = cap // page
        ids = rng.permutation(B * pages)
        table = torch.from_numpy(ids.reshape(B, pages).astype(np.int32)).cuda()

    def to_pool(x):
        if not page:
            return torch.from_numpy(x.copy()).cuda()
        p = x.reshape(B, H, pages, page, -1).transpose(0, 2, 1, 3, 4).reshape(B * pages, H, page, -1)
        pool = np.empty_like(p)
        pool[ids] = p
        return torch.from_numpy(pool).cuda()

    caches = [to_pool(x) for x in logical] + [None] * (2 - len(logical))
    wt = torch.full((B, H, T + 2), 9.0, device="cuda")
    wt[..., :T] = torch.from_numpy(w)
    tk, tn = torch.from_numpy(kept.astype(np.int32)).cuda(), torch.from_numpy(new.astype(np.int32)).cuda()
    tq.tq_evict_compact(caches[0], caches[1], tk, tn, T, weights=wt, block_table=table)
    for x, c in zip(logical, caches):
        assert torch.equal(c, to_pool(compact_reference(x, kept, new)))
    want = np.zeros((B, H, T), np.float32)
    for b in range(B):
        for h in range(H):
            want[b, h, :new[b]] = w[b, h, kept[b, h, :new[b]]]
    assert np.array_equal(wt[..., :T].cpu().numpy(), want)
    assert (wt[..., T:] == 9.0).all()
    again = [None if c is None else to_pool(x) for x, c in zip(logical + [None], caches)]
    tq.tq_evict_compact(again[0], again[1], tk, tn, T, block_table=table)      # without weights
    assert torch.equal(again[0], caches[0]) and (again[1] is None or torch.equal(again[1], caches[1]))


def test_compact_leaves_what_it_cannot_place(tq):
    """Indices outside j .. T - 1 and pages outside the pool: those tokens stay as they are."""
    cache = torch.arange(2 * 16 * 34, dtype=torch.int64, device="cuda").to(torch.uint8).view(1, 2, 16, 34).contiguous()
    before = cache.clone()
    kept = torch.tensor([[[0, 3, 16, 2, 9], [1, 2, 1 << 30, -5, 15]]], dtype=torch.int32, device="cuda")
    tq.tq_evict_compact(cache, None, kept, torch.tensor([5], dtype=torch.int32, device="cuda"), 16)
    want = before.clone()
    want[0, 0, 1], want[0, 0, 4] = before[0, 0, 3], before[0, 0, 9]
    want[0, 1, 0], want[0, 1, 1], want[0, 1, 4] = before[0, 1, 1], before[0, 1, 2], before[0, 1, 15]
    assert torch.equal(cache, want)
    pool = before.view(2, 2, 8, 34).clone()
    table = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")           # the second page is not in the pool
    k2 = torch.tensor([[[1, 9], [2, 10]]], dtype=torch.int32, device="cuda")
    tq.tq_evict_compact(pool, None, k2, torch.tensor([2], dtype=torch.int32, device="cuda"), 16, block_table=table)
    want = before.view(2, 2, 8, 34).clone()
    want[1, 0, 0], want[1, 1, 0] = want[1, 0, 1].clone(), want[1, 1, 2].clone()
    assert torch.equal(pool, want)
    tq.tq_evict_compact(pool, None, k2, torch.tensor([-3], dtype=torch.int32, device="cuda"), 16, block_table=table)
    assert torch.equal(pool, want)


def test_compact_of_a_repeated_index(tq):
    """The same index twice (not what the selection gives): both tokens take its block."""
    cache = torch.randint(0, 256, (1, 1, 2000, 66), dtype=torch.uint8, device="cuda")
    before = cache.clone()
    kept = torch.sort(torch.randint(700, 2000, (1, 1, 600), device="cuda")).values.int()
    kept[0, 0, 100:103] = kept[0, 0, 100]
    tq.tq_evict_compact(cache, None, kept, torch.tensor([600], dtype=torch.int32, device="cuda"), 2000)
    assert torch.equal(cache[0, 0, :600], before[0, 0][kept[0, 0].long()])
    assert torch.equal(cache[0, 0, 600:], before[0, 0, 600:])


def test_calls_on_two_streams_at_once(tq):
    """Two streams, each with its own workspace and cache, give what one stream gives."""
    rng = np.random.default_rng(8)
    T, keep = 3001, 1500
    blocks = [[torch.from_numpy(cache_of((2, 4, T + 7), n, rng)[0]).cuda() for n in (4, 2)] for _ in range(2)]
    qs = [torch.from_numpy(rng.standard_normal((2, 16, 128))).float().cuda() for _ in range(2)]
    books, signs = [tq.tq_codebook_load(128, n) for n in (4, 2)], tq.tq_signs_from_seed(workloads.SIGN_SEED)

    def chain(i, stream):
        with torch.cuda.stream(stream):
            k, v = (c.clone() for c in blocks[i])
            w, out = torch.zeros(2, 4, T, device="cuda"), torch.empty(2, 16, 128, device="cuda")
            ws = torch.empty(tq.tq_attn_weights_workspace_bytes(2, 16, 4, T), dtype=torch.uint8, device="cuda")
            kept = torch.empty(2, 4, keep, dtype=torch.int32, device="cuda")
            new = torch.empty(2, dtype=torch.int32, device="cuda")
            for _ in range(3):
                tq.tq_attn_decode_weights(qs[i], k, books[0], v, books[1], w, out, ws, T, SCALE, signs)
                tq.tq_evict_select(w, kept, new, T, 4, 100)
                tq.tq_evict_compact(k, v, kept, new, T, weights=w)
        return k, v, w, out, kept

    alone = [chain(i, torch.cuda.current_stream()) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    both = [chain(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------- together

def loop(tq, steps, graph, stream):
    """A decode loop with a budget: insert, attend, and once over the budget select and compact.
    Returns every step's outputs and the last state."""
    B, Hq, Hkv, T_cap, budget, first, last = 2, 8, 2, 64, 40, 2, 8
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(4)
    qkv = torch.randn(steps, B, Hq + 2 * Hkv, 128, generator=g, device=dev).to(torch.bfloat16)
    rope = tq.tq_rope_load(128, 1e6, sections=[16, 24, 24])
    kcb, vcb = tq.tq_codebook_load(128, 4), tq.tq_codebook_load(128, 3)
    signs = tq.tq_signs_from_seed(workloads.SIGN_SEED)
    kc = torch.zeros(B, Hkv, T_cap, 66, dtype=torch.uint8, device=dev)
    vc = torch.zeros(B, Hkv, T_cap, 50, dtype=torch.uint8, device=dev)
    w = torch.zeros(B, Hkv, T_cap, device=dev)
    lens = torch.tensor([0, 20], dtype=torch.int32, device=dev)    # the second has 20 tokens of nothing
    new = torch.empty_like(lens)
    kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device=dev)
    pos = torch.zeros(3, B, dtype=torch.int64, device=dev)
    x = torch.empty(B, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device=dev)
    q = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device=dev)
    out = torch.empty(B, Hq, 128, dtype=torch.float32, device=dev)
    ws = torch.empty(tq.tq_attn_weights_workspace_bytes(B, Hq, Hkv, T_cap), dtype=torch.uint8, device=dev)
    row = torch.arange(B, device=dev) * Hkv * T_cap

    def step():
        tq.tq_rope_apply(x[:, :Hq], pos, rope, q)
        tq.tq_insert_kv(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, rope, kcb, vcb, signs, kc, vc, row + lens, T_cap)
        lens.add_(1)
        tq.tq_attn_decode_weights(q, kc, kcb, vc, vcb, w, out, ws, T_cap, SCALE, signs, seq_lens=lens, decay=0.95)
        tq.tq_evict_select(w, kept, new, T_cap, first, last, seq_lens=lens)
        tq.tq_evict_compact(kc, vc, kept, new, T_cap, weights=w)
        lens.copy_(new)
        pos.add_(1)

    outs = []
    with torch.cuda.stream(stream):
        state = [kc, vc, w, lens, pos]
        start = [t.clone() for t in state]
        x.copy_(qkv[0])
        step()                                                     # first calls, before a capture
        for t, s in zip(state, start):
            t.copy_(s)
        torch.cuda.synchronize()
        if graph:
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg, stream=stream):
                step()
        for i in range(steps):
            x.copy_(qkv[i])
            cg.replay() if graph else step()
            outs.append(out.clone())
    torch.cuda.synchronize()
    return qkv, outs, [t.clone() for t in state]


def test_decode_loop(tq):
    """The loop eager, captured and replayed, and on another stream gives the same bits; and the plain loop over
    decoded vectors the same outputs (to the attention's tolerance at these sizes, 2^-10 of the largest)."""
    steps = 60
    qkv, outs, state = loop(tq, steps, False, torch.cuda.current_stream())
    for graph in (False, True):
        _, o2, s2 = loop(tq, steps, graph, torch.cuda.Stream())
        assert all(torch.equal(a, b) for a, b in zip(outs, o2)) and all(torch.equal(a, b) for a, b in zip(state, s2))

    from test_gpu_rope_insert import rotated
    B, Hq, Hkv, budget, first, last = 2, 8, 2, 40, 2, 8
    rope = tq.tq_rope_load(128, 1e6, sections=[16, 24, 24])
    s = oracle.sign_diagonal(workloads.SIGN_SEED)
    books = oracle_books()

    def kept_as(x, bits):
        idx, n, _ = codec.encode(x, s, books[bits][2])
        return codec.decode(idx, n, books[bits][0].astype(np.float32).astype(np.float64), s)

    k = [[[] for _ in range(Hkv)] for _ in range(B)]
    v = [[[] for _ in range(Hkv)] for _ in range(B)]
    w = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]
    for h in range(Hkv):
        k[1][h] = [np.zeros(128)] * 20
        v[1][h] = [np.zeros(128)] * 20
        w[1][h] = np.zeros(20)
    for i in range(steps):
        x = qkv[i].double().cpu().numpy()
        pos = np.full((3, B), i)
        turned = rotated(x, pos, rope)[0]
        q = torch.from_numpy(turned[:, :Hq]).to(torch.bfloat16).double().numpy()
        got = outs[i].double().cpu().numpy()
        for b in range(B):
            kn = kept_as(turned[b, Hq:Hq + Hkv], 4)
            vn = kept_as(x[b, Hq + Hkv:], 3)
            for h in range(Hkv):
                k[b][h].append(kn[h])
                v[b][h].append(vn[h])
                w[b][h] = np.append(w[b][h], 0.0) * 0.95
                for g in range(Hq // Hkv):
                    sc = SCALE * np.array(k[b][h]) @ q[b, h * 4 + g]
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    ref = p @ np.array(v[b][h])
                    assert np.abs(got[b, h * 4 + g] - ref).max() <= 2.0**-10 * max(1e-3, np.abs(ref).max()), (i, b, h, g)
                    w[b][h] += p
                if len(w[b][h]) > budget:
                    kept, _ = select_reference(w[b][h][None, None], None, budget, first, last)
                    at = kept[0, 0]
                    k[b][h] = [k[b][h][j] for j in at]
                    v[b][h] = [v[b][h][j] for j in at]
                    w[b][h] = w[b][h][at]
    lens = state[3].cpu().numpy()
    assert list(lens) == [budget, budget]
    for b in range(B):
        for h in range(Hkv):
            got = state[2][b, h].double().cpu().numpy()
            assert np.abs(got[:budget] - w[b][h]).max() <= 2.0**-14 and not got[budget:].any()


def test_one_row_of_any_strides(tq):
    """Strides of size-1 dimensions mean nothing: one row of weights, and one token of a cache."""
    T, keep = 100, 40
    w = torch.rand(T, 1, 1, device="cuda").permute(1, 2, 0)    # strides (1, 1, 1)
    assert w.stride()[2] == 1
    kept = [torch.empty(1, 1, keep, dtype=torch.int32, device="cuda") for _ in range(2)]
    for k, x in zip(kept, (w, w.clone(memory_format=torch.contiguous_format).view(1, 1, T))):
        tq.tq_evict_select(x, k, torch.empty(1, dtype=torch.int32, device="cuda"), T, 3, 5)
    assert torch.equal(kept[0], kept[1])
    cb, signs = tq.tq_codebook_load(128, 4), tq.tq_signs_from_seed(1)
    x = torch.randn(1, 5, 128, device="cuda").transpose(0, 1)  # [5, 1, 128], strides (128, 640, 1)
    blocks = [torch.empty(5, 66, dtype=torch.uint8, device="cuda") for _ in range(2)]
    tq.tq_encode_kv(x, cb, signs, blocks[0])
    tq.tq_encode_kv(x.reshape(5, 128).clone(), cb, signs, blocks[1])
    assert torch.equal(blocks[0], blocks[1])
