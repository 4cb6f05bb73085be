"""The calls that follow a step, on the GPU, against their plain 64-bit forms.

Verification returns whole numbers, which must be equal: both sides decide in
64 bits.  Weights are fp32; their bound counts the roundings (below).  The
accumulators must hold exactly the fp32 sums of the returned weights in the
order of the queries, and eviction copies bytes: both are compared exactly.
"""
import numpy as np
import pytest
import torch

import synth.workloads as W
from long_context_decode_csa2_b200 import csa2 as C
from long_context_decode_csa2_b200.decode import DecodeStep, FullCache, evict
from tests import _after_step as R
from tests._gpu import check_attention, dev, host

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SM = np.float32(1 / np.sqrt(512))


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

def _verify(target, draft, tokens, q_off, u, r, M=None, seq_len=None, ws=None, stream=None):
    B, V = len(q_off) - 1, target.shape[1]
    out = {"n": torch.full((B,), -7, dtype=torch.int32, device="cuda"),
           "t": torch.full((B,), -7, dtype=torch.int32, device="cuda"),
           "o": torch.full((B, M), -7, dtype=torch.int32, device="cuda") if M else None}
    ws = C.workspace(C.csa2_verify_drafts_workspace_bytes(B, V)) if ws is None else ws
    C.csa2_verify_drafts(target, _i32(tokens), _i32(q_off), u, r, out["n"], out["t"], ws, draft=draft,
                         out_tokens=out["o"], seq_len_in=seq_len, seq_len_out=seq_len, stream=stream)
    out["flags"] = C.device_status(ws)
    return out


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _check_verify(target, draft, tokens, q_off, u, r, flags=0, M=None):
    got = _verify(target, draft, tokens, q_off, u, r, M)
    n, t = R.verify(_f64(target), _f64(draft), np.asarray(tokens), np.asarray(q_off), _f64(u), _f64(r))
    assert np.array_equal(host(got["n"]), n), (host(got["n"]), n)
    assert np.array_equal(host(got["t"]), t), (host(got["t"]), t)
    assert got["flags"] == flags
    if M:
        for b, row in enumerate(host(got["o"])):
            lo, hi = int(q_off[b]), int(q_off[b + 1])
            want = [] if hi <= lo else [int(x) for x in np.asarray(tokens)[lo + 1:lo + 1 + n[b]]] + [int(t[b])]
            assert list(row) == (want + [-1] * M)[:M]
    return n, t


def _problem(B, n_hi, V, seed, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    counts = [(3 * b + seed) % (n_hi + 1) for b in range(B)] if B > 1 else [n_hi]
    off = np.concatenate([[0], np.cumsum(counts)])
    Q = max(1, int(off[-1]))
    z = torch.randn((Q, V), device="cuda", generator=g) * spread
    p = torch.softmax(z, 1)
    q = torch.softmax(z + 0.7 * torch.randn((Q, V), device="cuda", generator=g), 1)
    x = torch.multinomial(q, 1, generator=g)[:, 0].cpu().numpy()
    tokens = np.concatenate([x[:1], x[:-1]])
    return p, q, tokens, off, torch.rand(Q, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g)


@pytest.mark.parametrize("B,n_hi,V", [(1, 1, 1), (1, 5, 7), (3, 4, 1023), (2, 3, 1024), (5, 6, 1025), (4, 2, 8191),
                                      (1, 70, 300), (17, 9, 50001), (300, 3, 2049), (1, 4, 131072)])
@pytest.mark.parametrize("pt,qt", [("f32", "f32"), ("bf16", "f16"), ("f16", None), ("f32", None), ("f16", "bf16"),
                                   ("bf16", "f32")])
def test_verify_matches_the_plain_form(B, n_hi, V, pt, qt):
    p, q, tokens, off, u, r = _problem(B, n_hi, V, 5)
    _check_verify(p.to(DT[pt]), None if qt is None else q.to(DT[qt]), tokens, off, u, r, M=n_hi + 1)


@pytest.mark.parametrize("pt,qt", [("f32", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("lead", [1, 2, 3, 5])
def test_verify_rows_of_any_alignment_and_stride(pt, qt, lead):
    """Rows inside a wider tensor: their starts fall on every offset from a 16-byte border."""
    V = 4099
    p, q, tokens, off, u, r = _problem(6, 5, V, 9)
    wide = torch.full((p.shape[0], V + 13), float("nan"), device="cuda", dtype=DT[pt])   # a read past the row would show
    wide[:, lead:lead + V] = p.to(DT[pt])
    wq = torch.full((p.shape[0], V + 6), float("nan"), device="cuda", dtype=DT[qt])
    wq[:, 6 - lead:6 - lead + V] = q.to(DT[qt])
    _check_verify(wide[:, lead:lead + V], wq[:, 6 - lead:6 - lead + V], tokens, off, u, r, M=6)


@pytest.mark.parametrize("V,qt", [(262144, "bf16"), (300001, "f32"), (1000003, None)])
def test_verify_large_vocabularies(V, qt):
    """More partial sums than the scan keeps in registers."""
    p, q, tokens, off, u, r = _problem(2, 3, V, 6)
    _check_verify(p, None if qt is None else q.to(DT[qt]), tokens, off, u, r, M=4)
    last = torch.zeros((1, V), device="cuda")
    last[0, V - 1] = 0.5
    got = _verify(last, None, [0], [0, 1], u, torch.tensor([1.0], device="cuda"))
    assert list(host(got["t"])) == [V - 1]


def test_verify_many_sequences_of_a_large_vocabulary():
    """More partial sums per CTA than fit its shared memory: 700 sequences draw from one row of 300001 (stride 0)."""
    g = torch.Generator(device="cuda").manual_seed(2)
    V, B = 300001, 700
    row = torch.rand(V, device="cuda", generator=g) ** 4
    r = torch.rand(B, device="cuda", generator=g)
    got = _verify(row.expand(B, V), None, [0] * B, list(range(B + 1)), torch.zeros(B, device="cuda"), r)
    c = np.cumsum(_f64(row))
    assert np.array_equal(host(got["t"]), np.searchsorted(c, _f64(r) * c[-1], side="right")) and got["flags"] == 0


def test_verify_offsets_beyond_32_bits():
    """Rows 1.2e9 elements apart: element offsets above 2^31, byte offsets above 2^32."""
    V, far = 5003, 1_200_000_001
    p, q, tokens, off, u, r = _problem(1, 3, V, 4)
    big = torch.empty(2 * far + V, dtype=torch.bfloat16, device="cuda").as_strided((3, V), (far, 1))
    big.copy_(p.to(torch.bfloat16))
    _check_verify(big, q, tokens, off, u, r, M=3)
    _check_verify(p, big, tokens, off, torch.zeros(3, device="cuda"), r, M=3)


def test_verify_borders_are_exact():
    """Dyadic probabilities: every sum is exact, and a draw on a border takes the entry behind it."""
    V = 2500
    p = torch.zeros((8, V), device="cuda")
    p[:, [3, 1000, 1024, 2499]] = 0.25
    r = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.2499999, 1.0, 0.5], device="cuda")
    got = _verify(p, None, [0] * 8, list(range(9)), torch.zeros(8, device="cuda"), r)
    assert list(host(got["t"])) == [3, 1000, 1024, 2499, 2499, 3, 2499, 1024] and got["flags"] == 0
    _check_verify(p, None, [0] * 8, list(range(9)), torch.zeros(8, device="cuda"), r)
    odd = torch.tensor([float("nan"), -1.0, 1.5, float("inf")], device="cuda")
    got = _verify(p[:4], None, [0] * 4, list(range(5)), torch.zeros(4, device="cuda"), odd)
    assert list(host(got["t"])) == [3, 3, 2499, 2499]      # r outside [0, 1)
    # tests at the border: u q < p is strict
    p2 = torch.tensor([[0.25, 0.75], [0.5, 0.5]], device="cuda").repeat(4, 1)
    q2 = torch.tensor([[0.5, 0.5], [0.5, 0.5]], device="cuda").repeat(4, 1)
    u = torch.tensor([0.5, 0, 0.49999997, 0, 0.0, 0, 0.9999999, 0], device="cuda")
    n, t = _check_verify(p2, q2, [0, 0] * 4, [0, 2, 4, 6, 8], u, torch.full((4,), 0.3, device="cuda"))
    assert list(n) == [0, 1, 1, 0] and t[0] == 1


def test_verify_degenerate_distributions():
    V = 1100
    z = lambda: torch.zeros((2, V), device="cuda")  # noqa: E731
    u, r = torch.tensor([0.5, 0.0], device="cuda"), torch.tensor([0.6], device="cuda")

    def one(p, q, x, flags=0, u=u):
        return _check_verify(p, q, [0, x], [0, 2], u, r, flags=flags, M=2)

    p, q = z(), z()
    p[:, 7], q[:, 9] = 1.0, 1.0
    assert one(p, q, 9) == ([0], [7])                      # p = 0 at the draft: rejected, drawn from p
    assert one(p, q, 7)[0] == [1]                          # q = 0 at the draft, p > 0: stands
    same = torch.full((2, V), 1.0 / V, device="cuda")
    same[:, 5] = 0.0
    n, t = one(same, same, 5)                              # p = q and p = 0 at the draft: the residual is empty, p is drawn
    assert n == [0] and t[0] > 5
    assert one(z(), z(), 3, flags=32) == ([0], [-1])       # nothing to draw
    assert one(z(), None, 3, flags=32) == ([0], [-1])
    bad = torch.full((2, V), float("nan"), device="cuda")
    bad[:, 800:], bad[:, 20] = -1.0, 0.25
    assert one(bad, bad, 30)[1] == [20]                    # NaN and negative entries carry nothing
    sure = z()
    sure[:, 4] = 1.0
    assert one(sure, None, 4)[0] == [1]                    # greedy draft at probability 1
    assert one(sure, None, 5) == ([0], [4])
    more = z()
    more[0, 4], more[1, 8] = 2.0, 3.0                      # rows that do not sum to 1
    assert one(more, None, 6) == ([0], [4]) and one(more, None, 4) == ([1], [8])
    inf = z()
    inf[:, 11] = float("inf")
    got = _verify(inf, None, [0], [0, 1], u, r)
    assert list(host(got["t"])) == [11]


def test_verify_bad_tokens_and_offsets():
    p, q, tokens, off, u, r = _problem(1, 4, 900, 2)
    for x in (-1, 900, 2 ** 31 - 1):
        tok = tokens.copy()
        tok[2] = x
        n, _ = _check_verify(p, q, tok, off, torch.zeros(4, device="cuda"), r, flags=1)
        assert n[0] == 1
        _check_verify(p, None, tok, off, torch.zeros(4, device="cuda"), r, flags=1)
    for bad in ([0, 5], [-1, 3], [3, 2]):                  # beyond Q, negative, descending: no candidates
        got = _verify(p, q, tokens, bad, u, r, M=3)
        assert got["flags"] == 8 and list(host(got["n"])) == [0] and list(host(got["t"])) == [-1]
        assert list(host(got["o"])[0]) == [-1, -1, -1]
    got = _verify(p, q, tokens, [0, 4], torch.zeros(4, device="cuda"), r, M=2)   # the next token does not fit
    assert got["flags"] == 8 and list(host(got["o"])[0]) == list(tokens[1:3])
    none = _verify(p[:0], None, [], [0, 0], torch.zeros(0, device="cuda"), r)    # no query at all
    assert list(host(none["n"])) == [0] and list(host(none["t"])) == [-1] and none["flags"] == 0


def test_verify_rolls_lengths_back_and_its_workspace_is_reusable():
    p, q, tokens, off, u, r = _problem(9, 6, 3001, 4)
    n, t = R.verify(_f64(p), _f64(q), tokens, off, _f64(u), _f64(r))
    m = np.diff(off)
    ws = C.workspace(C.csa2_verify_drafts_workspace_bytes(9, 3001))
    for _ in range(3):
        ln = _i32(100 + np.arange(9))
        got = _verify(p, q, tokens, off, u, r, ws=ws, seq_len=ln)
        assert np.array_equal(host(ln), 100 + np.arange(9) - np.where(m > 0, m - 1 - n, 0))
        assert np.array_equal(host(got["t"]), t)


def test_verify_first_token_follows_the_target():
    """40000 sequences with one draft: the emitted token's frequencies are the target's (5 sigma; fixed seed)."""
    g = torch.Generator(device="cuda").manual_seed(8)
    B, p, q = 40000, np.array([.5, .25, .125, .125], np.float32), np.array([.1, .2, .3, .4], np.float32)
    x = torch.multinomial(torch.tensor(q, device="cuda"), B, replacement=True, generator=g).cpu().numpy()
    tokens = np.stack([np.zeros(B, int), x], 1).reshape(-1)
    row = lambda v: torch.tensor(v, device="cuda").expand(2 * B, 4)  # noqa: E731  (one row, stride 0)
    got = _verify(row(p), row(q), tokens, np.arange(B + 1) * 2, torch.rand(2 * B, device="cuda", generator=g),
                  torch.rand(B, device="cuda", generator=g))
    first = np.where(host(got["n"]) == 1, x, host(got["t"]))
    freq = np.bincount(first, minlength=4) / B
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / B))


# ---------------------------------------------------------------------------
# attention weights
# ---------------------------------------------------------------------------

def _rows(off, table, page):
    """row_of(sequence, positions) of either layout."""
    if table is None:
        return lambda b, t: off[b] + t
    return lambda b, t: table[b, t // page].astype(np.int64) * page + t % page


class WeightCase:
    """Seeded inputs of csa2_attn_weights: counts[b] queries of sequence b over lens[b] entries."""

    def __init__(self, lens, counts, k, page=0, seed=0, scale_lo=125, scale_hi=128, qscale=0.5, grouped=True):
        rng = np.random.default_rng(seed)
        self.lens, self.k, self.page = np.asarray(lens), k, page
        B, Q = len(lens), int(np.sum(counts))
        self.q_off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) if grouped else None
        self.q_seq = np.repeat(np.arange(B), counts)
        if page:
            need = (self.lens + page - 1) // page
            perm = rng.permutation(int(need.sum()) + 2).astype(np.int32)
            self.table = np.full((B, max(1, int(need.max()))), -1, np.int32)   # (unused entries are not read)
            o = 0
            for b, n in enumerate(need):
                self.table[b, :n] = perm[o:o + n]
                o += n
            self.off, self.rows = None, len(perm) * page
        else:
            cap = (self.lens + 7) // 8 * 8 + 8
            self.off = np.concatenate([[0], np.cumsum(cap)[:-1]]).astype(np.int64)
            self.table, self.rows = None, int(cap.sum())
        self.codes = rng.integers(0, 256, (self.rows, 256), dtype=np.uint8)
        self.scales = rng.integers(scale_lo, scale_hi, (self.rows, 16), dtype=np.uint8)
        self.q = torch.tensor(rng.standard_normal((Q, 16, 512)) * qscale).to(torch.bfloat16)
        self.topk = np.full((Q, k), -1, np.int32)
        for i in range(Q):
            L = int(self.lens[self.q_seq[i]])
            n = min(k, L)
            self.topk[i, :n] = np.sort(rng.choice(L, n, replace=False))
        self.acc = (rng.random(self.rows) * (rng.random(self.rows) < 0.5)).astype(np.float32)
        self.row_of = _rows(self.off, self.table, page)
        self.lse = np.zeros((Q, 16), np.float32)
        for i in range(Q):
            t = self.topk[i][self.topk[i] >= 0].astype(np.int64)
            if not len(t):
                self.lse[i] = -np.inf
                continue
            rows = self.row_of(self.q_seq[i], t)
            x = _f64(self.q)[i] @ R.dequant(self.codes[rows], self.scales[rows]).T * float(SM)
            m = x.max(1)
            self.lse[i] = m + np.log(np.exp(x - m[:, None]).sum(1)) + 0.2

    def call(self, n_acc=None, want_weights=True, acc=None, topk=None, ws=None, stream=None, lens=None):
        Q, B = len(self.topk), len(self.lens)
        d = {"acc": dev(self.acc if acc is None else acc),
             "w": torch.full((Q, self.k), -7.0, device="cuda") if want_weights else None}
        where = C.PageTable(dev(self.table), self.page) if self.page else dev(self.off)
        ws = C.workspace(C.csa2_attn_weights_workspace_bytes(B, Q, self.k)) if ws is None else ws
        C.csa2_attn_weights(self.q.cuda(), C.cache(dev(self.codes), dev(self.scales)), where,
                            _i32(self.lens if lens is None else lens), _i32(self.topk if topk is None else topk),
                            dev(self.lse), float(SM), d["acc"], ws, q_off=None if self.q_off is None else _i32(self.q_off),
                            n_accept=None if n_acc is None else _i32(n_acc), weights=d["w"], stream=stream)
        d["flags"] = C.device_status(ws)
        return d

    def counted(self, n_acc):
        first = np.concatenate([[0], np.cumsum(np.bincount(self.q_seq, minlength=len(self.lens)))])
        rank = np.arange(len(self.q_seq)) - first[self.q_seq]
        return np.ones(len(rank), bool) if n_acc is None else rank <= np.maximum(n_acc, 0)[self.q_seq]

    def check(self, n_acc=None, flags=0, topk=None):
        got = self.call(n_acc, topk=topk)
        assert got["flags"] == flags
        c = self.counted(n_acc)
        ids = self.topk if topk is None else topk
        want, A = R.weights(_f64(self.q), self.codes, self.scales, self.row_of, ids, self.lse, float(SM), self.q_seq, c)
        w = host(got["w"])
        # Roundings of a logit, each at most 2^-23 of A = sm_scale sum |q key|: a block's two MMAs of sixteen exact
        # products accumulate in fp32 (a truncation each at worst), sixteen scaled block sums are added (2^-24 each);
        # then x = s - lse (2^-24 |x|, |x| <= A + |lse|), expf (2 ulp = 2^-22), and sixteen positive terms (four adds
        # deep and one: 2^-24 each).  Weights below 2^-126, the
        # smallest normal number, are 0 by definition: an absolute 2^-126 (far-off scales give exp(-170) and less).
        lse = np.abs(np.where(np.isfinite(self.lse), self.lse, 0)).max(1)[:, None]
        tol = want * (48 * 2.0 ** -23 * A + 2.0 ** -24 * (A + lse) + 2.0 ** -22 + 5 * 2.0 ** -24) + 2.0 ** -126
        off = float(np.max(np.abs(w - want) / np.maximum(tol, 1e-300)))
        assert off <= 1, off
        # the accumulators: the returned weights, added in fp32 in the order of the queries
        acc = self.acc.copy()
        for i in np.nonzero(c)[0]:
            for j in np.nonzero(ids[i] >= 0)[0]:
                acc[self.row_of(self.q_seq[i], np.int64(ids[i, j]))] += w[i, j]
        assert np.array_equal(host(got["acc"]), acc)
        return got


@pytest.mark.parametrize("lens,k", [([1], 1), ([40], 64), ([300], 7), ([65], 65), ([0, 700, 8, 3000], 64),
                                    ([2048, 100, 5000], 2048), ([9001], 513)])
@pytest.mark.parametrize("page", [0, 512])
def test_weights_one_query_per_sequence(lens, k, page):
    WeightCase(lens, [1] * len(lens), k, page, seed=k, grouped=False).check()
    WeightCase(lens, [1] * len(lens), k, page, seed=k + 1).check()


@pytest.mark.parametrize("page", [0, 512, 1024])
@pytest.mark.parametrize("lens,counts,k", [([700, 90, 1500], [6, 0, 3], 64), ([1025], [33], 130), ([300] * 40, [2] * 40, 65),
                                           ([513, 2000], [1, 5], 300)])
def test_weights_of_candidates(lens, counts, k, page):
    c = WeightCase(lens, counts, k, page, seed=3)
    c.check()
    n = np.maximum(0, np.asarray(counts) - 2)
    got = c.check(n_acc=n)
    assert not host(got["w"])[~c.counted(n)].any()          # candidates that do not count weigh nothing
    c.check(n_acc=np.full(len(lens), 99))                   # more than there are: all
    c.check(n_acc=np.full(len(lens), -3))                   # fewer than none: the first
    again = c.call(n_acc=n)                                 # and the same bits every time
    assert torch.equal(again["acc"], got["acc"]) and torch.equal(again["w"], got["w"])
    bare = c.call(n_acc=n, want_weights=False)              # without the weights output
    assert torch.equal(bare["acc"], got["acc"])


@pytest.mark.parametrize("page,scale_lo,scale_hi,qscale", [(0, 125, 128, 0.5), (512, 125, 128, 0.5), (0, 221, 227, 1e-28)])
def test_weights_of_many_rows(page, scale_lo, scale_hi, qscale):
    """Enough rows that a warp takes two tiles at a time; the last case has scales of 2^97 in some rows."""
    c = WeightCase([3000, 700, 2000], [40, 0, 52], 1021, page, seed=11, scale_lo=scale_lo, scale_hi=scale_hi, qscale=qscale)
    assert 92 * 64 > 32 * 148
    c.check()
    c.check(n_acc=[38, 0, 50])


def test_weights_duplicates_and_positions_out_of_range():
    c = WeightCase([500, 800], [3, 2], 80, seed=5)
    ids = c.topk.copy()
    ids[:, 40:60] = ids[:, 20:40]                           # positions listed twice, out of order
    ids[1, 3:9] = -1                                        # empty slots in the middle
    c.check(topk=ids)
    ids[2, 0], ids[4, 79] = 500, 2 ** 31 - 1                # beyond the sequences
    got = c.call(topk=ids)
    assert got["flags"] == 1 and host(got["w"])[2, 0] == 0 and host(got["w"])[4, 79] == 0
    ids[2, 0], ids[4, 79] = -1, -1
    assert torch.equal(got["acc"], c.call(topk=ids)["acc"])
    # a length above the cache empties the sequence, as everywhere
    lens = np.array([500, c.rows + 1])
    far = c.call(lens=lens)
    assert far["flags"] & 2 and not host(far["w"])[3:].any()


@pytest.mark.parametrize("k", [64, 700])
@pytest.mark.parametrize("off", [[0, 3, 2], [0, 4, 7], [-1, 2, 5], [0, 6, 5]])
def test_weights_refuse_offsets_that_do_not_ascend(off, k):
    c = WeightCase([500, 800], [3, 2], k, seed=5)
    good = c.call()
    keep, c.q_off = c.q_off, np.array(off, np.int32)
    got = c.call()
    assert got["flags"] == 8 and not host(got["w"]).any() and np.array_equal(host(got["acc"]), c.acc)
    c.q_off = np.array([1, 3, 4], np.int32)                 # queries of no sequence weigh nothing
    got = c.call()
    w = host(got["w"])
    assert got["flags"] == 0 and not w[0].any() and not w[4].any() and w[1:4].all(1).sum() >= 1
    c.q_off = keep
    assert torch.equal(c.call()["acc"], good["acc"])


def test_weights_bad_page_is_skipped():
    c = WeightCase([1200, 600], [2, 1], 100, page=512, seed=6)
    good = host(c.call()["w"])
    c.table[0, 1] = 10 ** 6
    got = c.call()
    assert got["flags"] == 2
    hit = (c.q_seq[:, None] == 0) & (c.topk >= 512) & (c.topk < 1024)
    w = host(got["w"])
    assert not w[hit].any() and np.array_equal(w[~hit], good[~hit])
    changed = np.nonzero(host(got["acc"]) != c.acc)[0]
    ok = {int(c.table[b, t // 512]) * 512 + t % 512 for b, t in zip(c.q_seq.repeat(100), c.topk.reshape(-1))
          if t >= 0 and not (b == 0 and 512 <= t < 1024)}
    assert set(changed.tolist()) <= ok


@pytest.mark.parametrize("lo,hi,qscale", [(1, 4, 1e30), (250, 254, 1e-36), (0, 1, 1.0), (90, 165, 1e-3), (125, 128, 1e-30),
                                          (127, 128, 0.0)])
def test_weights_extreme_scales(lo, hi, qscale):
    """Block exponents and queries far outside fp16: both enter exactly."""
    c = WeightCase([200], [2], 64, seed=7, scale_lo=lo, scale_hi=hi, qscale=qscale)
    if qscale == 1e-3:                                      # logits up to 2^38: keep those whose exponentials exist
        c.lse[:] = np.float32(3e38)
        assert not host(c.call()["w"]).any()
        return
    c.check()


def test_weights_propagate_what_is_not_a_number():
    c = WeightCase([100], [1], 16, seed=8)
    c.lse[0, 3] = np.nan
    assert np.isnan(host(c.call()["w"])).all()
    c.lse[0, 3] = -np.inf                                   # a head without keys
    w = host(c.call()["w"])
    assert np.isfinite(w).all() and (w > 0).all()
    c.scales[c.topk[0, 2]] = 255                            # E8M0 NaN
    w = host(c.call()["w"])
    assert np.isnan(w[0, 2]) and np.isfinite(np.delete(w[0], 2)).all()


def test_weights_offsets_beyond_32_bits():
    """A sequence at the end of 20 million rows: byte offsets above 2^32 (5.1 GB of codes)."""
    rows, L, k = 20_000_000, 1000, 64
    c = WeightCase([L], [2], k, seed=9)
    codes = torch.empty((rows, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, 16), dtype=torch.uint8, device="cuda")
    acc = torch.zeros(rows, device="cuda")
    off = rows - 1000
    codes[off:], scales[off:], acc[off:] = dev(c.codes[:L]), dev(c.scales[:L]), dev(c.acc[:L])
    w = torch.zeros((2, k), device="cuda")
    ws = C.workspace(C.csa2_attn_weights_workspace_bytes(1, 2, k))
    C.csa2_attn_weights(c.q.cuda(), C.cache(codes, scales), torch.tensor([off], device="cuda"), _i32([L]), _i32(c.topk),
                        dev(c.lse), float(SM), acc, ws, q_off=_i32([0, 2]), weights=w)
    want = c.call()
    assert torch.equal(w, want["w"]) and torch.equal(acc[off:], want["acc"][:L]) and not acc[:off].any()


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

class EvictCase:
    def __init__(self, lens, acc_kind="mixed", page=0, idx=True, seed=0, room=None, spare=16):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.idx = np.asarray(lens), page, idx
        B = len(lens)
        if page:
            need = (self.lens + page - 1) // page
            room = need if room is None else np.asarray(room)
            perm = rng.permutation(int(need.sum() + room.sum()) + 1).astype(np.int32)   # one pool for both sides
            self.table = np.full((B, max(1, int(need.max()))), -1, np.int32)
            self.dtable = np.full((B, max(1, int(room.max()))), -1, np.int32)
            o = 0
            for b in range(B):
                self.table[b, :need[b]] = perm[o:o + need[b]]
                self.dtable[b, :room[b]] = perm[o + need[b]:o + need[b] + room[b]]
                o += need[b] + room[b]
            self.off = self.doff = None
            self.rows = self.drows = len(perm) * page
        else:
            cap = (self.lens + 7) // 8 * 8
            self.off = np.concatenate([[0], np.cumsum(cap)[:-1]]).astype(np.int64)
            self.rows = max(8, int(cap.sum()))
            dcap = cap + spare
            self.doff = np.concatenate([[0], np.cumsum(dcap)[:-1]]).astype(np.int64)
            self.drows = int(dcap.sum())
            self.table = self.dtable = None
        g = torch.Generator(device="cuda").manual_seed(seed)
        by = lambda r, w: torch.randint(0, 256, (r, w), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
        self.planes = [by(self.rows, 256), by(self.rows, 16)] + ([by(self.rows, 64), by(self.rows, 4)] if idx else [])
        self.dplanes = self.planes if page else [by(self.drows, p.shape[1]) for p in self.planes]
        a = rng.random(self.rows).astype(np.float32) ** 3
        if acc_kind == "mixed":
            a[rng.random(self.rows) < 0.6] = 0
        elif acc_kind == "zeros":
            a[:] = 0
        elif acc_kind == "ties":
            a = rng.integers(0, 3, self.rows).astype(np.float32) / 4
        elif acc_kind == "odd":
            a = rng.standard_normal(self.rows).astype(np.float32)
            pick = rng.random(self.rows)
            a[pick < .1], a[(pick > .1) & (pick < .2)] = np.nan, -0.0
            a[(pick > .2) & (pick < .25)], a[(pick > .25) & (pick < .3)] = np.inf, -np.inf
            a[(pick > .3) & (pick < .35)] = 1e-42
        self.acc = a
        self.row_of, self.drow_of = _rows(self.off, self.table, page), _rows(self.doff, self.dtable, page)

    def call(self, keep, max_keep, first=0, last=0, max_len=None, alias=False, ws=None, stream=None, dst=None, shift=0):
        B = len(self.lens)
        d = {"kept": torch.full((B, max_keep), -9, dtype=torch.int32, device="cuda"), "len": _i32(self.lens)}
        seq_len = d["len"] if alias else _i32(self.lens)
        src = self.planes
        dst = [p.clone() for p in self.dplanes] if dst is None else dst
        if self.page:
            src = dst                                        # one pool: source and destination pages of the same tensors
        acc = dev(np.concatenate([np.zeros(shift, np.float32), self.acc]))[shift:]
        dacc = acc if self.page else torch.full((self.drows,), -5.0, device="cuda")
        cache = lambda p: (C.cache(p[0], p[1]), C.cache(p[2], p[3]) if self.idx else None)  # noqa: E731
        (ms, is_), (md, id_) = cache(src), cache(dst)
        wh = (C.PageTable(dev(self.table), self.page), C.PageTable(dev(self.dtable), self.page)) if self.page else \
            (dev(self.off), dev(self.doff))
        max_len = int(max(self.lens.max(), 1)) if max_len is None else max_len
        ws = C.workspace(C.csa2_cache_evict_workspace_bytes(B, max_len)) if ws is None else ws
        C.csa2_cache_evict(ms, is_, acc, wh[0], seq_len, _i32(keep), max_len, max_keep, md, id_, dacc, wh[1], d["kept"],
                           d["len"], ws, first=first, last=last, stream=stream)
        d.update(dst=dst, acc=dacc, flags=C.device_status(ws))
        return d

    def check(self, keep, max_keep, first=0, last=0, flags=0, **kw):
        got = self.call(keep, max_keep, first, last, **kw)
        assert got["flags"] == flags
        kept, ln = host(got["kept"]), host(got["len"])
        want_planes = [p.clone() for p in self.dplanes]
        want_acc = self.acc.copy() if self.page else np.full(self.drows, -5.0, np.float32)
        for b, L in enumerate(self.lens):
            a = self.acc[self.row_of(b, np.arange(L))]
            pos = R.evict_positions(a, min(keep[b], max_keep), first, last)
            assert ln[b] == len(pos)
            assert np.array_equal(kept[b, :len(pos)], pos) and (kept[b, len(pos):] == -1).all()
            if len(pos):
                s = torch.from_numpy(self.row_of(b, pos)).cuda()
                t = torch.from_numpy(self.drow_of(b, np.arange(len(pos)))).cuda()
                for p, w in zip(self.planes, want_planes):
                    w[t] = p[s]
                want_acc[t.cpu().numpy()] = a[pos]
        for w, g in zip(want_planes, got["dst"]):
            assert torch.equal(w, g)                        # every other destination byte as it was
        assert np.array_equal(host(got["acc"]).view(np.int32), want_acc.view(np.int32))
        return got


@pytest.mark.parametrize("page", [0, 512])
@pytest.mark.parametrize("kind", ["mixed", "zeros", "ties", "odd"])
def test_evict_matches_the_plain_form(kind, page):
    lens = [0, 1, 7, 8, 9, 511, 512, 513, 4095, 4096, 4097, 9000]
    c = EvictCase(lens, kind, page, seed=len(kind))
    keep = [5, 1, 3, 8, 20, 100, 512, 200, 1, 2048, 4000, 4500]
    c.check(keep, 4500)
    c.check(keep, 4500, first=4, last=64)
    c.check(keep, 4500, first=100, last=0, alias=True)
    c.check([0] * 12, 16, first=3, last=3)                  # nothing stays
    c.check([-5] * 12, 1)
    c.check([10 ** 6] * 12, 9000)                           # everything stays
    c.check([3] * 12, 3, first=5, last=2)                   # fewer than are protected: the last ones, then the first
    c.check(keep, 4500, first=1, last=7, shift=3)           # accumulators off the 16-byte grid


@pytest.mark.parametrize("lens,keep", [([70001], 30000), ([300001, 5], 150000), ([1100000], 500001),
                                       ([200003] * 20 + [64] * 20, 70000)])
@pytest.mark.parametrize("kind", ["mixed", "zeros"])
def test_evict_long_sequences(lens, keep, kind):
    """Runs of positions longer than the shared memory that holds their keys, and every cluster size."""
    c = EvictCase(lens, kind, idx=False, seed=1)
    c.check([keep] * len(lens), keep, first=4, last=128, shift=len(lens) % 4)


@pytest.mark.parametrize("kind,share", [("ties", 0.2), ("ties", 0.5), ("ties", 0.9), ("odd", 0.3), ("odd", 0.6), ("odd", 0.85),
                                        ("odd", 0.97)])
@pytest.mark.parametrize("lens", [[70001, 9000], [900001]])
def test_evict_long_sequences_at_every_threshold(kind, share, lens):
    """Thresholds among many equal weights, among negative ones, and among NaN, over several CTAs."""
    c = EvictCase(lens, kind, idx=False, seed=3)
    c.check([int(n * share) for n in lens], max(lens), first=3, last=130)


@pytest.mark.parametrize("B", [1, 3, 10, 20, 40, 80, 200])
def test_evict_batches(B):
    c = EvictCase([(977 * (b + 1)) % 9001 for b in range(B)], "mixed", idx=B % 2 == 0, seed=B)
    c.check([(311 * (b + 2)) % 5000 for b in range(B)], 5000, first=1, last=8, max_len=20000)


def test_evict_nothing():
    EvictCase([0, 0], seed=1).check([3, 0], 4, first=1, last=1, max_len=0)
    EvictCase([0, 5], page=512, seed=1).check([0, 0], 1)


def test_evict_flags():
    c = EvictCase([1000, 600], "mixed", seed=2)
    c.check([900, 100], 300, last=10, flags=8)              # more than max_keep: cut to it
    c.doff = c.doff.copy()
    c.doff[1] = c.drows - 8                                 # the second sequence does not fit: left out
    got = c.call([300, 100], 300)
    assert got["flags"] == 2 and list(host(got["len"])) == [300, 0] and (host(got["kept"])[1] == -1).all()
    assert torch.equal(got["dst"][0][300:], c.dplanes[0][300:])
    c.doff[1] = 1004                                        # not a multiple of 8
    assert list(host(c.call([300, 100], 300)["len"])) == [300, 0]
    long = EvictCase([1000], "mixed", seed=3)
    got = long.call([50], 50, max_len=400)                  # a length above the bound is cut to it
    assert got["flags"] == 8 and list(host(got["kept"])[0]) == list(R.evict_positions(long.acc[:400], 50, 0, 0))
    p = EvictCase([2000, 900], "mixed", page=512, seed=4)
    p.dtable[0, 1] = 10 ** 6                                # a destination page outside the pool: its rows are not written
    before = [x.clone() for x in p.planes]
    got = p.call([1100, 300], 1100)
    assert got["flags"] == 2 and list(host(got["len"])) == [1100, 300]
    touched = torch.zeros(p.rows, dtype=torch.bool)
    for b, n in ((0, 1100), (1, 300)):
        pos = np.arange(n)
        pos = pos[(b == 1) | (pos < 512) | (pos >= 1024)]
        touched[torch.from_numpy(p.drow_of(b, pos))] = True
    same = (got["dst"][0] == before[0]).all(1).cpu()
    assert same[~touched].all()
    p.dtable[0, 1] = 3
    q = EvictCase([2000], "mixed", page=512, seed=5, room=[1])
    got = q.call([600], 600)                                # more than the destination's table holds
    assert got["flags"] == 2 and list(host(got["len"])) == [0]


def test_evict_offsets_beyond_32_bits():
    rows, L, n = 20_000_000, 3000, 1000
    codes = torch.empty((rows, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, 16), dtype=torch.uint8, device="cuda")
    dcodes, dscales = torch.empty_like(codes), torch.empty_like(scales)
    acc, dacc = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    off = rows - L
    g = torch.Generator(device="cuda").manual_seed(1)
    codes[off:] = torch.randint(0, 256, (L, 256), dtype=torch.uint8, device="cuda", generator=g)
    scales[off:] = torch.randint(0, 256, (L, 16), dtype=torch.uint8, device="cuda", generator=g)
    acc[off:] = torch.rand(L, device="cuda", generator=g)
    kept, ln = torch.zeros((1, n), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = C.workspace(C.csa2_cache_evict_workspace_bytes(1, L))
    at = torch.tensor([off], device="cuda")
    C.csa2_cache_evict(C.cache(codes, scales), None, acc, at, _i32([L]), _i32([n]), L, n, C.cache(dcodes, dscales), None,
                       dacc, at, kept, ln, ws)
    pos = R.evict_positions(host(acc[off:]), n, 0, 0)
    assert np.array_equal(host(kept)[0], pos) and C.device_status(ws) == 0
    at = torch.from_numpy(pos).cuda() + off
    assert torch.equal(dcodes[off:off + n], codes[at]) and torch.equal(dscales[off:off + n], scales[at])
    assert torch.equal(dacc[off:off + n], acc[at]) and not dacc[:off].any()


# ---------------------------------------------------------------------------
# graphs, streams
# ---------------------------------------------------------------------------

def test_calls_capture_and_replay():
    """One graph of all three calls, replayed on new inputs, and a second graph with its own workspaces."""
    p, q, tokens, off, u, r = _problem(4, 5, 5003, 3)
    wc = WeightCase([600, 900, 300, 70], np.diff(off), 64, seed=4)
    ec = EvictCase([600, 900, 300, 70], "mixed", seed=5)
    B, Q = 4, len(tokens)
    tok, qo, lens, keep = _i32(tokens), _i32(off), _i32([600, 900, 300, 70]), _i32([100, 300, 80, 70])
    n, t = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    acc, w = torch.zeros(wc.rows, device="cuda"), torch.zeros((Q, 64), device="cuda")
    eacc, dacc = dev(ec.acc), torch.zeros(ec.drows, device="cuda")
    kept, ln = torch.zeros((B, 300), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    wcache, woff, qd, ids, lse = C.cache(dev(wc.codes), dev(wc.scales)), dev(wc.off), wc.q.cuda(), _i32(wc.topk), dev(wc.lse)
    src = (C.cache(*ec.planes[:2]), C.cache(*ec.planes[2:]))
    dplanes = [x.clone() for x in ec.dplanes]
    dst = (C.cache(*dplanes[:2]), C.cache(*dplanes[2:]))
    so, do = dev(ec.off), dev(ec.doff)

    def go(ws):
        C.csa2_verify_drafts(p, tok, qo, u, r, n, t, ws[0], draft=q)
        C.csa2_attn_weights(qd, wcache, woff, lens, ids, lse, float(SM), acc, ws[1], q_off=qo, n_accept=n, weights=w)
        C.csa2_cache_evict(src[0], src[1], eacc, so, lens, keep, 900, 300, dst[0], dst[1], dacc, do, kept, ln, ws[2],
                           first=2, last=16)

    def spaces():
        return [C.workspace(b) for b in (C.csa2_verify_drafts_workspace_bytes(B, 5003),
                                         C.csa2_attn_weights_workspace_bytes(B, Q, 64),
                                         C.csa2_cache_evict_workspace_bytes(B, 900))]

    wa, wb = spaces(), spaces()
    go(wa)
    graphs = []
    for ws in (wa, wb):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            go(ws)
        graphs.append(g)
    for seed, g in enumerate(graphs * 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        u.copy_(torch.rand(Q, device="cuda", generator=gen))
        r.copy_(torch.rand(B, device="cuda", generator=gen))
        eacc.copy_(torch.rand(ec.rows, device="cuda", generator=gen))
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = R.verify(_f64(p), _f64(q), tokens, off, _f64(u), _f64(r))
        assert np.array_equal(host(n), want[0]) and np.array_equal(host(t), want[1])
        assert (host(w).sum(1) > 0).tolist() == wc.counted(want[0]).tolist()
        a = host(eacc)
        for b in range(B):
            pos = R.evict_positions(a[ec.row_of(b, np.arange(ec.lens[b]))], [100, 300, 80, 70][b], 2, 16)
            assert np.array_equal(host(kept)[b, :len(pos)], pos) and host(ln)[b] == len(pos)
    assert all(C.device_status(ws) == 0 for ws in wa + wb)


def test_decode_step_scratch_is_not_made_in_a_capture():
    """Scratch made there would be filled at the first replay only: the first verify and accumulate are plain calls."""
    p, q, tokens, off, u, r = _problem(3, 4, 5003, 3)
    wc = WeightCase([600, 900, 300], np.diff(off), 64, seed=4)
    Q, V = len(tokens), 5003
    step = DecodeStep("F", 3, 1024, 64, 64, queries=Q)
    step.topk[0].copy_(_i32(wc.topk))
    step.lse[0].copy_(dev(wc.lse))
    main = C.cache(dev(wc.codes), dev(wc.scales))
    caches = [FullCache(None, main, dev(wc.acc))]
    tok, qo, lens, woff, layers = _i32(tokens), _i32(off), _i32(wc.lens), dev(wc.off), [{"q": wc.q.cuda()}]
    narrow = torch.softmax(torch.randn((Q, 300), device="cuda"), 1)
    small = _i32(np.asarray(tokens) % 300)

    def verify(stream=None):
        return step.verify(p, tok, qo, u, r, draft=q, stream=stream)

    def accumulate(stream=None):
        step.accumulate(caches, woff, lens, layers, q_off=qo, n_accept=step.n_accept, stream=stream)

    def capture(call):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            call()
        return g

    step.verify(narrow, small, qo, u, r)                  # a small vocabulary first: a larger one needs more scratch
    for call in (verify, accumulate):
        with pytest.raises(ValueError, match="capture"):
            capture(call)
    want = R.verify(_f64(p), _f64(q), tokens, off, _f64(u), _f64(r))
    n, t = verify()
    assert np.array_equal(host(n), want[0]) and np.array_equal(host(t), want[1])
    accumulate()
    acc = caches[0].acc.clone()
    g = capture(lambda: (verify(), accumulate()))
    n.fill_(-9)
    caches[0].acc.copy_(dev(wc.acc))
    g.replay()
    assert np.array_equal(host(n), want[0]) and torch.equal(caches[0].acc, acc)
    step.verify(torch.softmax(torch.randn((Q, 60000), device="cuda"), 1), tok, qo, u, r)   # the graph keeps its own
    caches[0].acc.copy_(dev(wc.acc))
    g.replay()
    assert np.array_equal(host(n), want[0]) and torch.equal(caches[0].acc, acc) and step.device_flags() == 0


def test_one_workspace_serves_batches_of_any_size():
    """Large and small batches in turn on one workspace: neither's scratch lies where the other counts arrivals."""
    few, many = WeightCase([900] * 3, [6] * 3, 512, seed=1), WeightCase([70] * 150, [2] * 150, 64, seed=2)
    size = C.csa2_attn_weights_workspace_bytes
    ws = C.workspace(max(size(3, 18, 512), size(150, 300, 64)))
    cases = (few, many)
    want = [c.call()["acc"] for c in cases]
    for i in (0, 1, 0, 1):
        got = cases[i].call(want_weights=False, ws=ws)
        assert torch.equal(got["acc"], want[i]) and got["flags"] == 0
    a, b = _problem(2, 4, 131072, 3), _problem(140, 3, 5003, 4)
    size = C.csa2_verify_drafts_workspace_bytes
    ws = C.workspace(max(size(2, 131072), size(140, 5003)))
    for p, q, tokens, off, u, r in (a, b, a, b):
        got = _verify(p, q, tokens, off, u, r, ws=ws)
        n, t = R.verify(_f64(p), _f64(q), tokens, off, _f64(u), _f64(r))
        assert np.array_equal(host(got["n"]), n) and np.array_equal(host(got["t"]), t) and got["flags"] == 0


@pytest.mark.parametrize("B", [1023, 1024, 1025, 1100])
def test_more_sequences_than_arrival_counters(B):
    """Few queries over many sequences, most of them without any."""
    counts = np.zeros(B, np.int64)
    counts[[0, B // 2, B - 1]] = 3
    WeightCase(np.full(B, 40), counts, 32, seed=B).check()


def test_calls_on_two_streams_at_once():
    c1, c2 = WeightCase([900], [4], 128, seed=1), WeightCase([900], [4], 128, seed=2)
    e1, e2 = EvictCase([9000], seed=1), EvictCase([9000], seed=2)
    want = [c1.call(), c2.call(), e1.call([4000], 4000), e2.call([4000], 4000)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1, h1 = c1.call(stream=s1), e1.call([4000], 4000, stream=s1)
        with torch.cuda.stream(s2):
            g2, h2 = c2.call(stream=s2), e2.call([4000], 4000, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(g1["acc"], want[0]["acc"]) and torch.equal(g2["acc"], want[1]["acc"])
        for h, w in ((h1, want[2]), (h2, want[3])):
            assert torch.equal(h["kept"], w["kept"]) and all(torch.equal(a, b) for a, b in zip(h["dst"], w["dst"]))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_verification_step_then_accumulate_evict_and_decode():
    """As a serving loop uses them: a verification step over FRU layers, the candidates verified and the lengths rolled
    back, the standing candidates' attention accumulated, the caches cut to a budget, and a decode step over what is
    left, against the oracle on the rows that stayed."""
    import math

    import oracle

    pattern = "FRU"
    wl = W.DecodeWorkload("after_step", np.array([900, 4000, 2500]), pattern, P=64, k=64, needles=8, queries_per_seq=4)
    q_off, q_vis = wl.verify_queries()
    wq = W.DecodeWorkload("after_step_q", q_vis.astype(np.int64), pattern, P=64, k=64)
    layers_h = [W.layer_inputs_host(wq, l) for l in range(3)]
    Lc = W.layer_inputs_host(wl, 0)
    cache_h = W.full_cache_host(wl, 0, Lc["q_codes"], Lc["q_scales"])
    keys = ("q", "q_codes", "q_scales", "w", "win", "win_scale", "win_len")
    layers = [{k: dev(L[k]) for k in keys} for L in layers_h]
    rows = cache_h["idx_codes"].shape[0]
    planes = [dev(cache_h[k]) for k in ("idx_codes", "idx_scales", "main_codes", "main_scales")]
    src = FullCache(C.cache(*planes[:2]), C.cache(*planes[2:]), torch.zeros(rows, device="cuda"))
    off, lens = cache_h["seq_row_off"], wl.lengths.astype(np.int32)
    Q, B, V = len(q_vis), 3, 1000
    step = DecodeStep(pattern, B, wl.max_len, 64, 64, queries=Q)
    d_off, d_len, d_qoff = dev(off), dev(lens), dev(q_off)
    step.run([src], d_off, d_len, layers, q_off=d_qoff, q_vis=dev(q_vis))
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.softmax(torch.randn((Q, V), device="cuda", generator=g), 1)
    dr = torch.softmax(torch.log(p) + 0.3 * torch.randn((Q, V), device="cuda", generator=g), 1)
    tokens = torch.multinomial(dr, 1, generator=g)[:, 0].roll(1).int()
    u, r = torch.rand(Q, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g)
    n_acc, nxt = step.verify(p, tokens, d_qoff, u, r, draft=dr, seq_len=d_len)
    step.accumulate([src], d_off, d_len, layers, q_off=d_qoff, n_accept=n_acc)
    want_n, want_t = R.verify(_f64(p), _f64(dr), host(tokens), q_off, _f64(u), _f64(r))
    assert np.array_equal(host(n_acc), want_n) and np.array_equal(host(nxt), want_t)
    new_len = lens - (4 - 1 - want_n)
    assert np.array_equal(host(d_len), new_len)
    # every standing candidate's heads spread a mass of at most 1 each over selection and window
    acc = host(src.acc)
    counted = np.concatenate([np.arange(4) <= a for a in want_n])
    total = 0.0
    for l in range(3):
        ids, lse = host(step.topk[l]), host(step.lse[l])
        w, _ = R.weights(_f64(layers[l]["q"]), cache_h["main_codes"], cache_h["main_scales"],
                         lambda b, t: off[b] + t, ids, lse, 1 / math.sqrt(512), np.repeat(np.arange(B), 4), counted)
        total += w.sum()
    assert abs(acc.sum(dtype=np.float64) - total) <= 1e-5 * total and total < 3 * 16 * counted.sum()
    # cut to a budget; the recent window stays
    keep, max_keep = _i32([400, 1500, 3000]), 2500
    cap = [(int(n) + 7) // 8 * 8 + 8 for n in (400, 1500, 2500)]
    doff = np.array([0, cap[0], cap[0] + cap[1]], np.int64)
    dplanes = [torch.zeros((sum(cap), x.shape[1]), dtype=torch.uint8, device="cuda") for x in planes]
    dst = FullCache(C.cache(*dplanes[:2]), C.cache(*dplanes[2:]), torch.zeros(sum(cap), device="cuda"))
    kept = torch.zeros((B, max_keep), dtype=torch.int32, device="cuda")
    ws = C.workspace(C.csa2_cache_evict_workspace_bytes(B, wl.max_len))
    evict(src, dst, d_off, dev(doff), d_len, keep, wl.max_len, max_keep, kept, d_len, ws, first=4)
    left = host(d_len)
    assert list(left) == [400, 1500, new_len[2]] and C.device_status(ws) == 0
    small = {k: host(x) for k, x in zip(("idx_codes", "idx_scales", "main_codes", "main_scales"), dplanes)}
    for b in range(B):
        pos = R.evict_positions(acc[off[b]:off[b] + new_len[b]], [400, 1500, 3000][b], 4, 128)
        assert np.array_equal(host(kept)[b, :len(pos)], pos)
        for k, x in small.items():
            assert np.array_equal(x[doff[b]:doff[b] + len(pos)], cache_h[k][off[b] + pos])
    # the next decode step reads what is left
    wd = W.DecodeWorkload("after_step_d", left.astype(np.int64), pattern, P=64, k=64)
    dl_h = [W.layer_inputs_host(wd, l) for l in range(3)]
    dstep = DecodeStep(pattern, B, 2512, 64, 64)
    dl = [{k: dev(L[k]) for k in keys} for L in dl_h]
    dstep.run([dst], dev(doff), d_len, dl)
    small["seq_row_off"] = doff
    ref = oracle.decode_step(pattern, [small], doff, left, dl_h, 64, 64, 1 / math.sqrt(512))
    for l in range(3):
        assert np.array_equal(host(dstep.topk[l]), ref["topk"][l])
        check_attention(host(dstep.out[l]), ref["out"][l])
    dstep.accumulate([dst], dev(doff), d_len, dl)
    torch.cuda.synchronize()
    assert step.device_flags() == 0 and dstep.device_flags() == 0
