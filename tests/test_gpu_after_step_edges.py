"""Edges of the calls that follow a step, on the GPU, against the plain 64-bit
forms: what a batch, a distribution or a second use can bring that the tests of
each call's ordinary range do not."""
import numpy as np
import pytest
import torch

from long_context_decode_csa2_b200 import csa2 as C
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


# ---------------------------------------------------------------------------
# selection by pairs of CTAs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[1], [9, 2000, 1, 64], [4096] * 3])
def test_select_by_pairs_of_ctas_gives_what_one_gives(lens):
    """A large max_len gives every sequence two CTAs, of which short sequences leave the second one idle."""
    B, P, k = len(lens), 64, 128
    g = torch.Generator(device="cuda").manual_seed(B)
    by = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    idx = C.cache(by(0, 256, 4096 * B, 64), by(120, 130, 4096 * B, 4))
    q, qs, w = by(0, 256, B, 4, 64), by(120, 130, B, 4, 4), torch.rand((B, 4), device="cuda", generator=g)
    off = torch.arange(B, device="cuda") * 4096
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for max_len in (4096, 1 << 20, 1 << 20):
        pool, top = (torch.full((B, n), -9, dtype=torch.int32, device="cuda") for n in (P, k))
        ws = C.workspace(C.csa2_index_full_workspace_bytes(B, max_len, P, k))
        C.csa2_index_full(idx, q, qs, w, off, seq_len, max_len, P, k, pool, top, ws)
        assert C.device_status(ws) == 0
        got.append((pool, top))
    for pool, top in got[1:]:
        assert torch.equal(pool, got[0][0]) and torch.equal(top, got[0][1])
    assert [(r >= 0).sum().item() for r in got[0][1]] == [min(k, n) for n in lens]
