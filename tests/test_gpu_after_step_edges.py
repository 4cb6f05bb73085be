"""Edges of the calls that follow a step, on the GPU, against the plain 64-bit
forms: what a batch, a distribution or a second use can bring that the tests of
each call's ordinary range do not."""
import numpy as np
import pytest
import torch

from tests.test_gpu_after_step import EvictCase

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("max_len", [9000, 40000, 300000])
@pytest.mark.parametrize("page", [0, 512])
def test_evict_short_sequences_in_wide_clusters(max_len, page):
    """A cluster of up to 16 CTAs for sequences that give most of them no position at all: those reach the exchange of
    counts at once, whether or not the others run yet."""
    lens = [2, 3, 9, 64, 129, 700] if max_len > 9000 else [2, 3, 130, 2000]
    c = EvictCase(lens, "mixed", page, seed=max_len)
    keep = [max(1, n // 2) for n in lens]
    want = c.check(keep, 400, max_len=max_len, flags=8 if max(keep) > 400 else 0)   # 1000 of 2000 is cut to max_keep
    for _ in range(20):
        got = c.call(keep, 400, max_len=max_len)
        assert torch.equal(got["kept"], want["kept"]) and torch.equal(got["len"], want["len"])
