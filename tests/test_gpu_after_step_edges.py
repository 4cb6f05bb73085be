"""Edges of the calls that follow a step, on the GPU, against the plain 64-bit
forms: what a batch, a distribution or a second use can bring that the tests of
each call's ordinary range do not."""
import numpy as np
import math
import threading

import numpy as np
import pytest
import torch

import oracle
import synth.workloads as W
from long_context_decode_csa2_b200 import csa2 as C
from long_context_decode_csa2_b200.decode import DecodeStep, FullCache, evict
from tests import _after_step as R
from tests._gpu import check_attention, dev, host
from tests.test_gpu_after_step import SM, EvictCase, WeightCase, _check_verify, _f64, _i32, _verify

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("V", [5003, 131072, 300001])
def test_verify_draws_the_last_token_with_a_weight(V):
    """Filtered distributions end in zeros.  From r = 1 on the draw is the last token with a weight, whatever the sums
    round to; just below, it is the plain form's."""
    n = 100 if V > 200000 else 400
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(2.5 * torch.randn((n, V), device="cuda", generator=g), 1)
    end = torch.randint(1, V, (n,), device="cuda", generator=g)
    end[: n // 4] = torch.randint(1, min(V, 3000), (n // 4,), device="cuda", generator=g)
    p[torch.arange(V, device="cuda")[None] >= end[:, None]] = 0
    p[::3] *= (torch.rand((len(p[::3]), V), device="cuda", generator=g) < 0.01)   # few tokens stand
    p[torch.arange(n), end - 1] = 1e-3 * torch.rand(n, device="cuda", generator=g) + 1e-9
    u, off, tokens = torch.zeros(n, device="cuda"), list(range(n + 1)), [0] * n
    for r in (1.0, 1.5, float("inf")):
        got = _verify(p, None, tokens, off, u, torch.full((n,), r, device="cuda"))
        assert torch.equal(got["t"].long(), end - 1) and got["flags"] == 0, r
    _check_verify(p, None, tokens, off, u, torch.full((n,), 1 - 2.0 ** -24, device="cuda"))
    _check_verify(p, None, tokens, off, u, torch.rand(n, device="cuda", generator=g))
    # drawn from a residual: rejected at candidate 1, which the target never takes
    q = p * (0.2 + torch.rand(p.shape, device="cuda", generator=g))
    q[torch.arange(n), end - 1] = 0
    p2, q2 = (torch.stack([x, x], 1).reshape(2 * n, V) for x in (p, q))
    got = _verify(p2, q2, [0, V - 1] * n, list(range(0, 2 * n + 1, 2)), torch.zeros(2 * n, device="cuda"),
                  torch.ones(n, device="cuda"))
    want = torch.where(end == V, 1, 0)                       # (a draft at V - 1 stands where the target has it)
    assert torch.equal(got["n"].long(), want) and torch.equal(got["t"].long(), end - 1) and got["flags"] == 0


# ---------------------------------------------------------------------------
# attention weights
# ---------------------------------------------------------------------------

def _lse(c):
    """The log-sum-exps of a case whose rows or queries were changed."""
    for i, ids in enumerate(c.topk):
        rows = c.row_of(c.q_seq[i], ids[ids >= 0].astype(np.int64))
        x = c.q[i].double().numpy() @ R.dequant(c.codes[rows], c.scales[rows]).T * float(SM)
        m = x.max(1)
        c.lse[i] = m + np.log(np.exp(x - m[:, None]).sum(1)) + 0.2


@pytest.mark.parametrize("lens,counts,k", [([300, 500], [2, 1], 64), ([3000, 2000], [40, 52], 1021)])
@pytest.mark.parametrize("empty", ["codes", "query"])
def test_weights_of_rows_with_scales_far_apart(lens, counts, k, empty):
    """Blocks of 2^97 and more that add nothing (their codes are zero, or the query there is), beside blocks of 2^-97 to
    2^-64 under queries that bring those to ordinary logits: the large scale must not touch the small ones."""
    c = WeightCase(lens, counts, k, seed=3)
    rng = np.random.default_rng(4)
    c.scales[:] = rng.integers(30, 45, c.scales.shape)
    c.q = (c.q.float() * 2.0 ** 85).to(torch.bfloat16)
    big = rng.random(c.scales.shape) < 0.1
    big[:, 5] = rng.random(len(big)) < 0.8                  # rows without a large scale among them
    if empty == "query":
        big[:, :5], big[:, 6:] = False, False
        c.q[:, :, 160:192] = 0
    else:
        c.codes.reshape(-1, 16, 16)[big] = rng.choice(np.array([0x00, 0x80, 0x08, 0x88], np.uint8), (big.sum(), 16))
    c.scales[big] = rng.integers(224, 255, int(big.sum()))
    _lse(c)
    c.check()


@pytest.mark.parametrize("lo,lens,counts,k", [(31, [300, 500], [2, 1], 64), (33, [300, 500], [2, 1], 64),
                                              (36, [300], [1], 64), (31, [3000, 2000], [40, 52], 1021),
                                              (34, [3000, 2000], [40, 52], 1021)])
def test_weights_of_queries_with_a_wide_range(lo, lens, counts, k):
    """The largest elements of each query row meet zero codes, so that elements of 2^-(lo-4) to 2^-lo of them decide.
    Down to 2^-31 they enter exactly and the ordinary bound holds; below, each enters within 2^-39 of the largest."""
    c = WeightCase(lens, counts, k, seed=5)
    rng = np.random.default_rng(6)
    shape = (len(c.q), 16, 512)
    x = rng.integers(128, 256, shape) / 128 * np.exp2(3.0 - rng.integers(3, 8, shape)) * rng.choice([-1.0, 1.0], shape)
    x /= 2                                                  # 2^-5 to 1
    x[:, :, 64:96] = 2.0 ** (lo - 5)
    c.q = torch.tensor(x).to(torch.bfloat16)
    assert np.array_equal(_f64(c.q), x)                     # (they are bf16 numbers)
    c.codes[:, 32:48] = rng.choice(np.array([0x00, 0x80, 0x08, 0x88], np.uint8), (c.rows, 16))
    _lse(c)
    top = np.abs(x).max(2)                                  # of a head's row
    tiny = np.abs(x) < top[:, :, None] * 2.0 ** -31
    assert tiny.any() == (lo > 31)
    if lo == 31:
        c.check()
        return
    got = c.call()
    want, A = R.weights(x, c.codes, c.scales, c.row_of, c.topk, c.lse, float(SM), c.q_seq, c.counted(None))
    # the ordinary roundings (tests of the call's range), and 2^-39 of the largest for every product of a small element
    extra = np.zeros_like(want)
    for i, ids in enumerate(c.topk):
        key = np.abs(R.dequant(c.codes[c.row_of(c.q_seq[i], ids)], c.scales[c.row_of(c.q_seq[i], ids)]))
        extra[i] = (2.0 ** -39 * top[i][:, None] * (tiny[i].astype(np.float64) @ key.T)).max(0) * float(SM)
    lse = np.abs(c.lse).max(1)[:, None]
    tol = want * (48 * 2.0 ** -23 * A + 2.0 ** -24 * (A + lse) + 2.0 ** -22 + 5 * 2.0 ** -24) + 2.0 ** -126
    tol += want * np.expm1(extra)
    assert got["flags"] == 0 and np.all(np.abs(host(got["w"]) - want) <= tol)


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


def test_evict_from_two_threads():
    """Two threads, each with its own stream, buffers and workspace, evict sequences of different lengths: neither's
    launch depends on what the other one's asked of the kernel."""
    cases = [EvictCase([700000], "mixed", idx=False, seed=1), EvictCase([30000], "mixed", idx=False, seed=2)]
    want = [c.call([500], 500)["kept"] for c in cases]
    errors = []

    def work(c, want):
        stream, ws = torch.cuda.Stream(), C.workspace(256)
        src, dst = C.cache(*c.planes), C.cache(*[p.clone() for p in c.dplanes])
        acc, dacc, off, doff = dev(c.acc), torch.zeros(c.drows, device="cuda"), dev(c.off), dev(c.doff)
        n, kept, ln, L = _i32([500]), torch.zeros((1, 500), dtype=torch.int32, device="cuda"), _i32([0]), _i32(c.lens)
        torch.cuda.synchronize()
        try:
            for _ in range(3000):
                C.csa2_cache_evict(src, None, acc, off, L, n, int(c.lens[0]), 500, dst, None, dacc, doff, kept, ln, ws,
                                   stream=stream)
            stream.synchronize()
            assert torch.equal(kept, want) and C.device_status(ws) == 0
        except Exception as e:  # noqa: BLE001  (reported by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def _by_rows(rows, planes, g):
    return [torch.randint(0, 256, (rows, p.shape[1]), dtype=torch.uint8, device="cuda", generator=g) for p in planes]


@pytest.mark.parametrize("page", [0, 512])
@pytest.mark.parametrize("n,kind,share,shift,lens", [
    (2, "mixed", 0.3, 0, [0, 1, 9, 513, 9000]), (3, "ties", 0.6, 3, [700, 4097]), (4, "odd", 0.9, 0, [5000, 129]),
    (2, "odd", 0.97, 1, [70001]), (3, "mixed", 0.5, 0, [900001, 64]), (5, "zeros", 0.4, 2, [3000])])
def test_evict_layers_matches_the_plain_form(n, kind, share, shift, lens, page):
    """Every layer keeps the entries with the largest sum of the layers' weights, whatever each layer's own are."""
    cases = [EvictCase(lens, kind, page, seed=7 * l + n) for l in range(n)]
    c0, B, first, last = cases[0], len(lens), 3, 70
    keep = [int(L * share) for L in lens]
    max_keep, rows, drows = max(max(keep), 1), c0.rows, c0.drows
    g = torch.Generator(device="cuda").manual_seed(n)
    src = [[p.clone() for p in c.planes] for c in cases]
    dst = src if page else [_by_rows(drows, c.planes, g) for c in cases]
    before = [[p.clone() for p in d] for d in dst]
    acc = [dev(np.concatenate([np.zeros(shift, np.float32), c.acc]))[shift:] for c in cases]
    dacc = acc if page else [torch.full((drows,), -5.0, device="cuda") for _ in cases]
    where = (C.PageTable(dev(c0.table), page), C.PageTable(dev(c0.dtable), page)) if page else (dev(c0.off), dev(c0.doff))
    seq_len, kept = _i32(lens), torch.full((B, max_keep), -9, dtype=torch.int32, device="cuda")
    ws = C.workspace(C.csa2_cache_evict_workspace_bytes(B, max(lens)))
    mains, idxs = ([C.cache(*p[i:i + 2]) for p in src] for i in (0, 2))
    dmains, didxs = ([C.cache(*p[i:i + 2]) for p in dst] for i in (0, 2))
    C.csa2_cache_evict_layers(mains, idxs, acc, where[0], seq_len, _i32(keep), max(lens), max_keep, dmains, didxs, dacc,
                              where[1], kept, seq_len, ws, first=first, last=last)   # the lengths in place
    assert C.device_status(ws) == 0
    with np.errstate(invalid="ignore"):
        total = cases[0].acc.copy()
        for c in cases[1:]:
            total = total + c.acc                            # fp32, layer by layer
    want_acc = [c.acc.copy() if page else np.full(drows, -5.0, np.float32) for c in cases]
    for b, L in enumerate(lens):
        at = c0.row_of(b, np.arange(L))
        pos = R.evict_positions(total[at], keep[b], first, last)
        assert host(seq_len)[b] == len(pos)
        assert np.array_equal(host(kept)[b, :len(pos)], pos) and (host(kept)[b, len(pos):] == -1).all()
        if len(pos):
            s, t = c0.row_of(b, pos), c0.drow_of(b, np.arange(len(pos)))
            for l, c in enumerate(cases):
                want_acc[l][t] = c.acc[s]
                for p, w in zip(c.planes, before[l]):
                    w[torch.from_numpy(t).cuda()] = p[torch.from_numpy(s).cuda()]
    for l in range(n):
        assert all(torch.equal(w, d) for w, d in zip(before[l], dst[l])), l
        assert np.array_equal(host(dacc[l]).view(np.int32), want_acc[l].view(np.int32)), l


def test_evict_layers_with_shared_accumulators():
    """Layers that add to the same accumulators: they count once and are moved once for all."""
    c = EvictCase([3000, 700], "odd", seed=1)
    one = c.call([1500, 200], 1500, first=2, last=30)
    acc, dacc, w = dev(c.acc), torch.full((c.drows,), -5.0, device="cuda"), C.workspace(256)
    kept, ln = torch.zeros((2, 1500), dtype=torch.int32, device="cuda"), _i32([0, 0])
    dst = [[p.clone() for p in c.dplanes] for _ in range(3)]
    C.csa2_cache_evict_layers([C.cache(*c.planes[:2])] * 3, None, [acc] * 3, dev(c.off), _i32(c.lens), _i32([1500, 200]),
                              3000, 1500, [C.cache(*d[:2]) for d in dst], None, [dacc] * 3, dev(c.doff), kept, ln, w,
                              first=2, last=30)
    assert C.device_status(w) == 0
    assert torch.equal(kept, one["kept"]) and torch.equal(ln, one["len"])
    assert np.array_equal(host(dacc).view(np.int32), host(one["acc"]).view(np.int32))
    for d in dst:
        assert all(torch.equal(a, b) for a, b in zip(d[:2], one["dst"][:2]))
        assert all(torch.equal(a, b) for a, b in zip(d[2:], c.dplanes[2:]))   # no indexer cache was given


def test_evict_layers_captured_and_replayed():
    """One graph of two layers' eviction on a side stream, replayed over changing accumulators and lengths."""
    a, b = EvictCase([5000, 300], seed=1), EvictCase([5000, 300], seed=2)
    acc = [dev(a.acc), dev(b.acc)]
    dst = [[p.clone() for p in c.dplanes] for c in (a, b)]
    dacc = [torch.zeros(a.drows, device="cuda") for _ in range(2)]
    src, keep = [C.cache(*c.planes[:2]) for c in (a, b)], _i32([1000, 60])
    at, to, mains = dev(a.off), dev(a.doff), [C.cache(*d[:2]) for d in dst]
    seq_len, ln, kept = _i32([5000, 300]), _i32([0, 0]), torch.zeros((2, 1000), dtype=torch.int32, device="cuda")
    ws = C.workspace(C.csa2_cache_evict_workspace_bytes(2, 5000))

    def go():
        C.csa2_cache_evict_layers(src, None, acc, at, seq_len, keep, 5000, 1000, mains, None, dacc, to, kept, ln, ws,
                                  first=1, last=9)

    go()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="thread_local"):
        go()
    for turn, lens in enumerate(([5000, 300], [4097, 12], [9, 300])):
        g = torch.Generator(device="cuda").manual_seed(turn)
        seq_len.copy_(_i32(lens))
        for x in acc:
            x.copy_(torch.rand(len(x), device="cuda", generator=g))
        graph.replay()
        total = host(acc[0]) + host(acc[1])
        for s, L in enumerate(lens):
            pos = R.evict_positions(total[a.row_of(s, np.arange(L))], [1000, 60][s], 1, 9)
            assert host(ln)[s] == len(pos) and np.array_equal(host(kept)[s, :len(pos)], pos)
            for c, d, x, y in zip((a, b), dst, acc, dacc):
                rows, there = torch.from_numpy(a.row_of(s, pos)).cuda(), torch.from_numpy(a.drow_of(s, np.arange(len(pos)))).cuda()
                assert torch.equal(d[0][there], c.planes[0][rows]) and torch.equal(y[there], x[rows])
    assert C.device_status(ws) == 0


@pytest.mark.parametrize("page", [0, 512])
def test_decode_after_eviction_of_two_full_layers(page):
    """FRUFR: the second Full layer selects inside the first one's pool on its own caches.  Its accumulators differ from
    the first one's; after the eviction both hold the same tokens at the same positions, so that the next step agrees
    with the oracle on the rows that stayed."""
    pattern, P, k = "FRUFR", 64, 64
    wl = W.DecodeWorkload("evict_two", np.array([900, 5000, 2500]), pattern, P=P, k=k, needles=8)
    layers_h = [W.layer_inputs_host(wl, l) for l in range(len(pattern))]
    fulls = wl.full_layers()
    caches_h = [W.full_cache_host(wl, f, layers_h[f]["q_codes"], layers_h[f]["q_scales"]) for f in fulls]
    names = ("idx_codes", "idx_scales", "main_codes", "main_scales")
    off, lens, B = caches_h[0]["seq_row_off"], wl.lengths.astype(np.int32), 3
    rows = caches_h[0]["idx_codes"].shape[0]
    keys = ("q", "q_codes", "q_scales", "w", "win", "win_scale", "win_len")
    layers = [{n: dev(L[n]) for n in keys} for L in layers_h]
    left = [300, 1250, 2000]
    if page:
        # source rows as pages of a pool, the destination's pages behind them
        need, dneed = [(int(n) + page - 1) // page for n in lens], [(n + page - 1) // page for n in left]
        table, dtable = np.full((B, max(need)), -1, np.int32), np.full((B, max(need)), -1, np.int32)
        perm = np.random.default_rng(2).permutation(sum(need) + sum(dneed)).astype(np.int32)
        o = 0
        for b in range(B):
            table[b, :need[b]], o = perm[o:o + need[b]], o + need[b]
            dtable[b, :dneed[b]], o = perm[o:o + dneed[b]], o + dneed[b]
        row_of = lambda b, t: table[b, t // page].astype(np.int64) * page + t % page  # noqa: E731
        drow_of = lambda b, t: dtable[b, t // page].astype(np.int64) * page + t % page  # noqa: E731
        src_rows, dst_rows, rows = C.PageTable(dev(table), page), C.PageTable(dev(dtable), page), len(perm) * page
    else:
        cap = [(n + 7) // 8 * 8 for n in left]
        doff = np.concatenate([[0], np.cumsum(cap)[:-1]]).astype(np.int64)
        row_of, drow_of = lambda b, t: off[b] + t, lambda b, t: doff[b] + t
        src_rows, dst_rows = dev(off), dev(doff)
    planes = []
    for c in caches_h:
        by = []
        for n in names:
            p = np.zeros((rows, c[n].shape[1]), np.uint8)
            for b in range(B):
                p[row_of(b, np.arange(lens[b]))] = c[n][off[b]:off[b] + lens[b]]
            by.append(dev(p))
        planes.append(by)
    full = lambda p, r: FullCache(C.cache(*p[:2]), C.cache(*p[2:]), torch.zeros(r, device="cuda"))  # noqa: E731
    src = [full(p, rows) for p in planes]
    step = DecodeStep(pattern, B, 5120, P, k)
    d_len = dev(lens)
    step.run(src, src_rows, d_len, layers)
    step.accumulate(src, src_rows, d_len, layers)
    acc = [host(c.acc) for c in src]
    if page:
        dplanes, dst = planes, src
    else:
        dplanes = [[torch.zeros((sum(cap), p.shape[1]), dtype=torch.uint8, device="cuda") for p in ps] for ps in planes]
        dst = [full(p, sum(cap)) for p in dplanes]
    kept = torch.zeros((B, 2000), dtype=torch.int32, device="cuda")
    ws = C.workspace(C.csa2_cache_evict_workspace_bytes(B, 5120))
    with pytest.raises(ValueError, match="2 Full layers"):
        evict(src[1], dst[1], src_rows, dst_rows, d_len, _i32(left), 5120, 2000, kept, d_len, ws)
    evict(src, dst, src_rows, dst_rows, d_len, _i32(left), 5120, 2000, kept, d_len, ws, first=4)
    assert host(d_len).tolist() == left and C.device_status(ws) == 0
    small, alone = [{n: np.zeros((6000, caches_h[0][n].shape[1]), np.uint8) for n in names} for _ in fulls], []
    soff = np.array([0, 1000, 3000], np.int64)
    for b in range(B):
        at = row_of(b, np.arange(lens[b]))
        pos = R.evict_positions(acc[0][at] + acc[1][at], left[b], 4, 128)
        assert np.array_equal(host(kept)[b, :left[b]], pos)
        alone += [not np.array_equal(pos, R.evict_positions(a[at], left[b], 4, 128)) for a in acc]
        for f, c in enumerate(caches_h):
            for i, n in enumerate(names):
                small[f][n][soff[b]:soff[b] + left[b]] = c[n][off[b] + pos]
                got = host(dplanes[f][i])
                assert np.array_equal(got[drow_of(b, np.arange(left[b]))], c[n][off[b] + pos]), (b, f, n)
            t = drow_of(b, np.arange(left[b]))
            assert np.array_equal(host(dst[f].acc)[t], acc[f][row_of(b, pos)])
    assert any(alone)                                     # a layer by itself would have kept others
    wd = W.DecodeWorkload("evict_two_d", np.array(left), pattern, P=P, k=k)
    nl_h = [W.layer_inputs_host(wd, l) for l in range(len(pattern))]
    nl = [{n: dev(L[n]) for n in keys} for L in nl_h]
    step.run(dst, dst_rows, d_len, nl)
    ref = oracle.decode_step(pattern, small, soff, np.array(left, np.int32), nl_h, P, k, 1 / math.sqrt(512))
    for l in range(len(pattern)):
        assert np.array_equal(host(step.topk[l]), ref["topk"][l]), l
        check_attention(host(step.out[l]), ref["out"][l])
    assert step.device_flags() == 0


# ---------------------------------------------------------------------------
# accumulators of new entries
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("page", [0, 512])
def test_acc_clear_clears_the_new_entries_only(page):
    old, new = [0, 5, 700, 510, 9, 30, -3, 8], [1, 5, 4000, 1030, 3, 31, 6, 8]
    B = len(old)
    rng = np.random.default_rng(3)
    if page:
        need = [(max(n, 1) + page - 1) // page for n in new]
        perm = rng.permutation(sum(need) + 2).astype(np.int32)
        table = np.full((B, max(need)), -1, np.int32)
        at = np.concatenate([[0], np.cumsum(need)])
        for b in range(B):
            table[b, :need[b]] = perm[at[b]:at[b + 1]]
        row_of, rows = (lambda b, t: table[b, t // page].astype(np.int64) * page + t % page), len(perm) * page
        where = C.PageTable(dev(table), page)
    else:
        cap = [(max(n, 1) + 7) // 8 * 8 for n in new]
        off = np.concatenate([[0], np.cumsum(cap)[:-1]]).astype(np.int64)
        row_of, rows, where = (lambda b, t: off[b] + t), sum(cap), dev(off)
    acc = rng.random(rows).astype(np.float32)
    want = acc.copy()
    for b in range(B):
        want[row_of(b, np.arange(max(old[b], 0), max(new[b], 0)))] = 0
    d, ws = dev(acc), C.workspace(C.csa2_acc_clear_workspace_bytes(B))
    C.csa2_acc_clear(d, where, _i32(old), _i32(new), ws)
    assert np.array_equal(host(d), want) and C.device_status(ws) == 0
    # what does not fit is left alone: a sequence that ends behind the rows, entries of a page that does not exist
    d = dev(acc)
    if page:
        table[2, 1], want = 10 ** 6, acc.copy()
        C.csa2_acc_clear(d, C.PageTable(dev(table), page), _i32(old), _i32([0] * 2 + [1300] + [0] * 5), ws)
        want[row_of(2, np.arange(1024, 1300))] = 0
    else:
        want = acc
        C.csa2_acc_clear(d, where, _i32(old), _i32([0] * 7 + [9]), ws)
    assert C.device_status(ws) == 2 and np.array_equal(host(d), want)


@pytest.mark.parametrize("page", [0, 512])
def test_entries_appended_after_an_eviction_start_without_weight(page):
    """Two caches (or two sets of a pool's pages) used in turn: what an entry's row carried before the eviction is not
    the entry's.  A captured step appends, attends and accumulates between two evictions."""
    import synth

    lens0, left, room, k = [900, 333], [400, 100], 40, 64
    wl = W.DecodeWorkload("recycled", np.array(lens0), "FU", P=64, k=k, ratio=2, room=room)
    layers_h = [W.layer_inputs_host(wl, l) for l in range(2)]
    c = W.full_cache_host(wl, 0, layers_h[0]["q_codes"], layers_h[0]["q_scales"])
    off, B = c["seq_row_off"], 2
    layers = [{n: dev(L[n]) for n in ("q", "q_codes", "q_scales", "w", "win", "win_scale", "win_len")} for L in layers_h]
    names = ("idx_codes", "idx_scales", "main_codes", "main_scales")
    planes = [dev(c[n]) for n in names]
    if page:
        rows = 8 * page
        row_of = lambda tab, b, t: tab[b, t // page].astype(np.int64) * page + t % page  # noqa: E731
        tabs = np.array([[0, 5], [3, -1]], np.int32), np.array([[2, 7], [6, -1]], np.int32)
        pool = [torch.zeros((rows, p.shape[1]), dtype=torch.uint8, device="cuda") for p in planes]
        for b in range(B):
            t = np.arange(lens0[b])
            for p, q in zip(pool, planes):
                p[torch.from_numpy(row_of(tabs[0], b, t)).cuda()] = q[torch.from_numpy(off[b] + t).cuda()]
        caches = [FullCache(C.cache(*pool[:2]), C.cache(*pool[2:]), torch.zeros(rows, device="cuda"))] * 2
        where = [C.PageTable(dev(t), page) for t in tabs]
        row = [lambda b, t, tab=tab: row_of(tab, b, t) for tab in tabs]
    else:
        rows = len(c["idx_codes"])
        make = lambda ps: FullCache(C.cache(*ps[:2]), C.cache(*ps[2:]), torch.zeros(rows, device="cuda"))  # noqa: E731
        caches = [make(planes), make([torch.zeros_like(p) for p in planes])]
        where, row = [dev(off)] * 2, [lambda b, t: off[b] + t] * 2
    step = DecodeStep("FU", B, 1000, 64, k, ratio=2, projection=False)
    seq_len = _i32(lens0)
    tok = lambda t: dict(  # noqa: E731
        raw=dev(synth.normal_bf16(91, synth.T_RAW, t, 0, B * 512).reshape(B, 512)),
        logit=dev(synth.normal_f32(91, synth.T_LOGITS, t, 0, B)),
        idx_raw=dev(synth.normal_bf16(91, synth.T_IDXRAW, t, 0, B * 128).reshape(B, 128)))
    ws, kept = C.workspace(256), torch.zeros((B, 400), dtype=torch.int32, device="cuda")
    caches[1].acc.fill_(0.0) if page else caches[1].acc.fill_(7.0)   # the second cache has been used before
    if page:                                                # and so have the pool's free pages
        free = sorted(set(range(8)) - {0, 5, 3})
        for f in free:
            caches[0].acc[f * page:(f + 1) * page] = 7.0
    side = 0
    for turn in range(3):
        cache, rows_now = caches[side], where[side]
        if turn == 1:                                       # the graph replays the same calls
            token = tok(0)
            graph = step.capture([cache], rows_now, seq_len, layers, new_tokens=[token])
        before = host(seq_len).copy()
        for b in range(B):                                  # rows behind the end may carry anything
            cache.acc[torch.from_numpy(row[side](b, np.arange(before[b], before[b] + 3))).cuda()] = 3.0
        kept_acc = [host(cache.acc)[row[side](b, np.arange(before[b]))] for b in range(B)]
        want = [np.concatenate([a, np.zeros(3, np.float32)]) for a in kept_acc]
        for t in range(6):
            new = tok(10 * turn + t)
            if turn == 1:
                for n, x in new.items():
                    token[n].copy_(x)
                graph.replay()
            else:
                step.run([cache], rows_now, seq_len, layers, new_tokens=[new])
            step.accumulate([cache], rows_now, seq_len, layers)
            # the entries' weights, layer by layer, in fp32
            for l in range(2):
                w, probe = torch.zeros((B, k), device="cuda"), torch.zeros_like(cache.acc)
                C.csa2_attn_weights(layers[l]["q"], cache.main, rows_now, seq_len, step.topk[l], step.lse[l],
                                    step.sm_scale, probe, step.ws_weights, weights=w)
                for b in range(B):
                    ids = host(step.topk[l])[b]
                    want[b][ids[ids >= 0]] += host(w)[b][ids >= 0]
        now = host(seq_len)
        assert now.tolist() == [n + 3 for n in before]
        for b in range(B):
            got = host(cache.acc)[row[side](b, np.arange(now[b]))]
            assert np.array_equal(got, want[b]), (turn, b)
        if turn < 2:
            evict(cache, caches[1 - side], rows_now, where[1 - side], seq_len, _i32(left), 1000, 400, kept, seq_len, ws,
                  first=2, last=16)
            pos = [R.evict_positions(want[b], left[b], 2, 16) for b in range(B)]
            for b in range(B):
                assert np.array_equal(host(kept)[b, :left[b]], pos[b])
            side = 1 - side
    assert step.device_flags() == 0 and C.device_status(ws) == 0


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


# ---------------------------------------------------------------------------
# offsets near the end of 64 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("far", [2 ** 63 - 8, 2 ** 63 - 512, 2 ** 40])
def test_offsets_whose_sum_wraps_are_outside(far):
    """A row offset so large that its sum with the length is negative: the sequence is left out and flagged."""
    c = EvictCase([300, 700], "mixed", seed=1)
    good = c.call([100, 200], 200)
    for side in ("off", "doff"):
        keep, at = getattr(c, side), getattr(c, side).copy()
        at[0] = far
        setattr(c, side, at)
        got = c.call([100, 200], 200)
        assert got["flags"] == 2 and host(got["len"]).tolist() == [0, 200]
        assert torch.equal(got["kept"][1], good["kept"][1]) and (got["kept"][0] == -1).all()
        setattr(c, side, keep)
    w = WeightCase([300, 700], [2, 2], 64, seed=2)
    full, w.off = w.call(), np.array([far, w.off[1]])
    got = w.call()
    assert got["flags"] == 3 and not host(got["w"])[:2].any() and torch.equal(got["w"][2:], full["w"][2:])
    acc, ws = torch.ones(64, device="cuda"), C.workspace(256)
    C.csa2_acc_clear(acc, torch.tensor([far, 32], device="cuda"), _i32([0, 0]), _i32([16, 8]), ws)
    assert C.device_status(ws) == 2 and acc.sum() == 56 and not acc[32:40].any()
    g = torch.Generator(device="cuda").manual_seed(1)
    by = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    idx = C.cache(by(0, 256, 4096, 64), by(120, 130, 4096, 4))
    pool, top = (torch.full((2, n), -9, dtype=torch.int32, device="cuda") for n in (64, 64))
    ws = C.workspace(C.csa2_index_full_workspace_bytes(2, 2048, 64, 64))
    C.csa2_index_full(idx, by(0, 256, 2, 4, 64), by(120, 130, 2, 4, 4), torch.rand((2, 4), device="cuda", generator=g),
                      torch.tensor([far, 2048], device="cuda"), _i32([1000, 1000]), 2048, 64, 64, pool, top, ws)
    assert C.device_status(ws) == 2 and (top[0] == -1).all() and (top[1] >= 0).all()
