"""Refusals of the rotary, weighted attention and eviction calls at the edges
of what they allow: host code only, nothing is enqueued."""

import pytest

from test_rope_evict_cpu import UNSUPPORTED, _attend, _select, tq  # noqa: F401


@pytest.mark.parametrize("keep", [(1 << 30) + 1, 2**31 - 8192, 2**31 - 1])
def test_select_refuses_more_kept_than_it_can_index(tq, keep):  # noqa: F811
    """The kernel's index past the last kept token (a cluster's 8192 threads further) has to fit 32 bits."""
    assert _select(tq, keep=keep) == UNSUPPORTED


def test_attend_refuses_contexts_past_32_bits(tq):  # noqa: F811
    """Positions a round past the context's end have to fit 32 bits; the longest context still has a workspace."""
    longest = 2**31 - 8192
    assert tq.tq_attn_weights_workspace_bytes(1, 1, 1, longest) > 4 * longest
    for T in (longest + 1, 2**31 - 32, 2**31 - 8, 2**31 - 1):
        assert tq.tq_attn_weights_workspace_bytes(1, 1, 1, T) == 0
        assert _attend(tq, Hq=2, T=T, T_cap=2**31 - 8, ws=2**32, bytes=1 << 50) == (UNSUPPORTED if T <= 2**31 - 8 else -1)
