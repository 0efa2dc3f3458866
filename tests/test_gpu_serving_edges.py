"""Rotary insert, weighted attention and eviction at the edges of what their
calls allow."""

import numpy as np
import pytest
import torch

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
