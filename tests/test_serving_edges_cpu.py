"""Refusals of the rotary, weighted attention and eviction calls at the edges
of what they allow: host code only, nothing is enqueued."""

import pytest

from test_rope_evict_cpu import UNSUPPORTED, _select, tq  # noqa: F401


@pytest.mark.parametrize("keep", [(1 << 30) + 1, 2**31 - 8192, 2**31 - 1])
def test_select_refuses_more_kept_than_it_can_index(tq, keep):  # noqa: F811
    """The kernel's index past the last kept token (a cluster's 8192 threads further) has to fit 32 bits."""
    assert _select(tq, keep=keep) == UNSUPPORTED
