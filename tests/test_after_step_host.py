"""The calls that follow a step, without a GPU: host-side checks of the C
entry points and the binding (bad arguments are refused before any launch),
the orchestration in DecodeStep, and the plain forms the GPU tests use."""
import gc
import weakref

import numpy as np
import pytest
import torch

from long_context_decode_csa2_b200 import csa2 as C
from long_context_decode_csa2_b200.decode import DecodeStep, FullCache, evict
from tests import _after_step as R
from tests.test_binding_host import FakeStream, fake  # noqa: F401  (fixture)

FAKE = 0x100000


def _cache(rows=1024, codes=FAKE, scales=FAKE):
    return C.MXFP4Cache(codes, scales, rows)


# ---------------------------------------------------------------------------
# C entry points: refusals on the host
# ---------------------------------------------------------------------------

def _verify(target=FAKE, tt=0, ts=100, draft=FAKE, dt=0, ds=100, tokens=FAKE, q_off=FAKE, u=FAKE, r=FAKE, B=2, Q=6,
            V=100, li=None, lo=None, na=FAKE, nt=FAKE, out=None, M=0, ws=FAKE, wn=1 << 20):
    return C.lib().csa2_verify_drafts(target, tt, ts, draft, dt, ds, tokens, q_off, u, r, B, Q, V, li, lo, na, nt, out,
                                      M, ws, wn, None)


@pytest.mark.parametrize("bad,rc", [
    (dict(B=-1), -1), (dict(Q=-1), -1), (dict(V=0), -1), (dict(V=(1 << 30) + 1), -1),
    (dict(target=None), -1), (dict(tokens=None), -1), (dict(u=None), -1), (dict(r=None), -1), (dict(q_off=None), -1),
    (dict(na=None), -1), (dict(nt=None), -1), (dict(ws=None), -1), (dict(ws=FAKE + 128), -1),
    (dict(tt=3), -1), (dict(tt=-1), -1), (dict(dt=7), -1),
    (dict(target=FAKE + 2), -1),                  # fp32 rows off their 4-byte grid
    (dict(tt=1, target=FAKE + 1), -1),            # bf16 rows off their 2-byte grid
    (dict(draft=FAKE + 2), -1), (dict(ts=-1), -1), (dict(ds=-5), -1),
    (dict(li=FAKE), -1), (dict(lo=FAKE), -1),     # the lengths go together
    (dict(out=FAKE, M=0), -1), (dict(wn=255), -3), (dict(B=0), 0),
])
def test_verify_refuses(bad, rc):
    assert _verify(**bad) == rc
    if rc:
        assert C.lib().csa2_last_error().startswith(b"csa2_verify_drafts")


def _weights(q=FAKE, cache=None, off=FAKE, ln=FAKE, q_off=FAKE, n_acc=None, topk=FAKE, k=64, lse=FAKE, acc=FAKE,
             w=None, B=2, Q=6, ws=FAKE, wn=1 << 20):
    return C.lib().csa2_attn_weights(q, cache or _cache(), off, ln, q_off, n_acc, topk, k, lse, 0.1, acc, w, B, Q, ws,
                                     wn, None)


@pytest.mark.parametrize("bad,rc", [
    (dict(k=0), -1), (dict(k=2049), -1), (dict(Q=-1), -1), (dict(B=0), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -1),
    (dict(off=None), -1), (dict(ln=None), -1), (dict(topk=None), -1), (dict(lse=None), -1), (dict(acc=None), -1),
    (dict(ws=None), -1), (dict(ws=FAKE + 16), -1), (dict(cache=C.MXFP4Cache(FAKE, FAKE, 1001)), -1),
    (dict(q_off=None), -1),                       # one query per sequence means Q == B
    (dict(q_off=None, Q=2, n_acc=FAKE), -1),      # accepted counts need q_off
    (dict(wn=256 + 256 + 6 * 64 * 4 - 1), -3), (dict(Q=0), 0),
])
def test_weights_refuses(bad, rc):
    assert _weights(**bad) == rc


def test_weights_paged_refuses():
    L = C.lib()

    def call(rows=2048, pages=FAKE, page_rows=512, max_pages=4):
        return L.csa2_attn_weights_paged(FAKE, _cache(rows), pages, page_rows, max_pages, FAKE, None, None, FAKE, 64, FAKE,
                                         0.1, FAKE, None, 2, 2, FAKE, 16, None)

    assert call(page_rows=768) == -1 and call(page_rows=256) == -1 and call(rows=1000) == -1
    assert call(pages=None) == -1 and call(max_pages=0) == -1
    assert call() == -3


def _evict(main=None, idx=None, acc=FAKE, off=FAKE, ln=FAKE, keep=FAKE, dmain=None, didx=None, dacc=None, doff=FAKE,
           kept=FAKE, lo=FAKE, B=2, max_len=512, max_keep=256, first=0, last=0, ws=FAKE, wn=256):
    far = 1 << 30  # the destination: other memory
    none = C.MXFP4Cache(None, None, 0)
    return C.lib().csa2_cache_evict(main or _cache(1024, 1 << 24, 1 << 25), idx or none, acc, off, ln, keep,
                                    dmain or _cache(1024, far, far + (1 << 24)), didx or none,
                                    dacc if dacc is not None else far + (1 << 26), doff, kept, lo, B, max_len, max_keep,
                                    first, last, ws, wn, None)


@pytest.mark.parametrize("bad,rc", [
    (dict(B=-1), -1), (dict(off=None), -1), (dict(doff=None), -1), (dict(ln=None), -1), (dict(keep=None), -1),
    (dict(acc=None), -1), (dict(dacc=0), -1), (dict(kept=None), -1), (dict(lo=None), -1), (dict(ws=None), -1),
    (dict(ws=FAKE + 4), -1), (dict(max_len=-1), -1), (dict(max_keep=0), -1), (dict(first=-1), -1), (dict(last=-2), -1),
    (dict(main=C.MXFP4Cache(FAKE, FAKE, 1001)), -1),
    (dict(idx=C.MXFP4Cache(FAKE, FAKE, 1024)), -1),                        # an indexer source without a destination
    (dict(dmain=C.MXFP4Cache(1 << 24, 1 << 28, 1024)), -1),                # the same codes on both sides
    (dict(dmain=C.MXFP4Cache((1 << 24) + 1023 * 256, 1 << 28, 1024)), -1),  # the last source row is the first destination row
    (dict(dacc=FAKE + 1023 * 4), -1),
    (dict(B=65536), -2), (dict(wn=255), -3), (dict(B=0), 0),
])
def test_evict_refuses(bad, rc):
    assert _evict(**bad) == rc


def test_evict_paged_refuses():
    none = C.MXFP4Cache(None, None, 0)

    def call(rows=2048, page_rows=512, max_pages=4, dmax=2, dpages=FAKE):
        c = _cache(rows)
        return C.lib().csa2_cache_evict_paged(c, none, FAKE, FAKE, max_pages, FAKE, FAKE, c, none, FAKE, dpages, dmax,
                                              page_rows, FAKE, FAKE, 2, 512, 256, 0, 0, FAKE, 16, None)

    assert call(page_rows=500) == -1 and call(rows=1032) == -1 and call(max_pages=0) == -1 and call(dmax=0) == -1
    assert call(dpages=None) == -1
    assert call() == -3


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------

def _verify_args(Q=6, B=2, V=50):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(target=torch.zeros((Q, V)), tokens=i(Q), q_off=i(B + 1), u=torch.zeros(Q), r=torch.zeros(B),
                n_accept=i(B), next_tok=i(B), ws=torch.zeros(4096, dtype=torch.uint8), draft=torch.zeros((Q, V)),
                out_tokens=i(B, 4))


@pytest.mark.parametrize("name,bad", [
    ("target", torch.zeros((6, 50), dtype=torch.float64)), ("target", torch.zeros((5, 50))),
    ("target", torch.zeros((50, 6)).t()),                     # a row's probabilities are not contiguous
    ("target", torch.zeros(300)), ("draft", torch.zeros((6, 49))), ("draft", torch.zeros((6, 50), dtype=torch.int32)),
    ("tokens", torch.zeros(6, dtype=torch.int64)), ("q_off", torch.zeros(2, dtype=torch.int32)),
    ("u", torch.zeros(5)), ("r", torch.zeros(2, dtype=torch.float64)), ("next_tok", torch.zeros(1, dtype=torch.int32)),
    ("out_tokens", torch.zeros(8, dtype=torch.int32)), ("out_tokens", torch.zeros((1, 8), dtype=torch.int32)),
])
def test_verify_binding_checks(fake, name, bad):  # noqa: F811
    args = _verify_args()
    args[name] = bad
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_verify_drafts(**args)
    assert e.value.status == -1 and name in str(e.value) and not fake.calls
    wide = torch.zeros((6, 64))
    C.csa2_verify_drafts(**{**_verify_args(), "target": wide[:, 3:53], "draft": torch.zeros((6, 50), dtype=torch.float16)})
    (_, a), = fake.calls
    assert a[:3] == (wide.data_ptr() + 12, 0, 64) and a[4:6] == (2, 50) and a[10:13] == (2, 6, 50) and a[18] == 4


def test_weights_and_evict_binding_checks(fake):  # noqa: F811
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    main, idx = C.cache(z(64, 256), z(64, 16)), C.cache(z(64, 64), z(64, 4))
    off, ws = torch.zeros(2, dtype=torch.int64), z(256)
    base = dict(q=torch.zeros((2, 16, 512), dtype=torch.bfloat16), main_kv=main, seq_row_off=off, seq_len=i(2),
                topk=i(2, 8), lse=torch.zeros((2, 16)), sm_scale=0.1, acc=torch.zeros(64), ws=ws)
    for name, bad in (("acc", torch.zeros(63)), ("lse", torch.zeros((2, 15))), ("weights", torch.zeros((2, 7))),
                      ("q_off", i(2)), ("q", torch.zeros((2, 16, 512), dtype=torch.float16))):
        with pytest.raises(C.Csa2Error, match=name):
            C.csa2_attn_weights(**{**base, name: bad})
    pt = C.PageTable(i(2, 1), 512)
    ev = dict(main_src=main, idx_src=idx, acc_src=torch.zeros(64), src=off, seq_len=i(2), keep=i(2), max_len=32,
              max_keep=16, main_dst=main, idx_dst=idx, acc_dst=torch.zeros(64), dst=off, kept=i(2, 16),
              seq_len_out=i(2), ws=ws)
    for change in (dict(dst=pt), dict(src=pt), dict(src=pt, dst=C.PageTable(i(2, 1), 1024)), dict(idx_dst=None),
                   dict(kept=i(2, 15)), dict(acc_src=torch.zeros(60)), dict(keep=torch.zeros(2))):
        with pytest.raises(C.Csa2Error):
            C.csa2_cache_evict(**{**ev, **change})
    assert not fake.calls
    C.csa2_attn_weights(**base)
    C.csa2_attn_weights(**{**base, "seq_row_off": pt})
    C.csa2_cache_evict(**ev)
    C.csa2_cache_evict(**{**ev, "src": pt, "dst": pt, "idx_src": None, "idx_dst": None})
    assert [n for n, _ in fake.calls] == ["csa2_attn_weights", "csa2_attn_weights_paged", "csa2_cache_evict",
                                          "csa2_cache_evict_paged"]


def test_bindings_refuse_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        C.csa2_verify_drafts(**_verify_args())


def test_decode_step_orchestrates_the_calls(fake):  # noqa: F811
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    caches = [FullCache(C.cache(z(64, 64), z(64, 4)), C.cache(z(64, 256), z(64, 16)), torch.zeros(64))
              for _ in range(2)]
    step = DecodeStep("FRFU", 2, 32, 16, 8, device="cpu", concurrent=False, queries=5)
    layers = [dict(q=torch.zeros((5, 16, 512), dtype=torch.bfloat16)) for _ in range(4)]
    off, q_off, lens = torch.zeros(2, dtype=torch.int64), i(3), i(2)
    n_acc, nxt = step.verify(torch.zeros((5, 40)), i(5), q_off, torch.zeros(5), torch.zeros(2), seq_len=lens)
    step.accumulate(caches, off, lens, layers, q_off=q_off, n_accept=n_acc)
    names = [n for n, _ in fake.calls]
    assert names == ["csa2_verify_drafts"] + ["csa2_attn_weights"] * 4
    a = fake.calls[0][1]
    assert a[13] == a[14] == lens.data_ptr() and a[15] == n_acc.data_ptr() and a[16] == nxt.data_ptr()
    for layer, f in enumerate((0, 0, 1, 1)):                      # every layer adds to its Full layer's accumulators
        a = fake.calls[1 + layer][1]
        assert a[1] is caches[f].main and a[10] == caches[f].acc.data_ptr()
        assert a[6] == step.topk[layer].data_ptr() and a[8] == step.lse[layer].data_ptr()
        assert a[4] == q_off.data_ptr() and a[5] == n_acc.data_ptr()
    with pytest.raises(ValueError, match="q_off"):
        step.accumulate(caches, off, lens, layers)
    with pytest.raises(ValueError, match="acc"):
        step.accumulate([FullCache(c.idx, c.main) for c in caches], off, lens, layers, q_off=q_off)
    with pytest.raises(ValueError, match="verification"):
        DecodeStep("F", 2, 32, 16, 8, device="cpu", concurrent=False).verify(torch.zeros((5, 40)), i(5), q_off,
                                                                             torch.zeros(5), torch.zeros(2))
    with pytest.raises(ValueError, match="acc"):
        evict(FullCache(caches[0].idx, caches[0].main), caches[1], off, off, lens, i(2), 32, 16, i(2, 16), i(2), z(256))


def test_decode_step_keeps_its_scratch(fake, monkeypatch):  # noqa: F811
    """A captured graph goes on using the scratch that it was captured with: a larger vocabulary adds to it."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    made, real = [], C.workspace
    need = {40: 512, 400: 4096}

    def record(nbytes, device=None):
        ws = real(nbytes, device)
        made.append(weakref.ref(ws))
        return ws

    step = DecodeStep("F", 2, 32, 16, 8, device="cpu", concurrent=False, queries=5)
    monkeypatch.setattr(C, "workspace", record)
    monkeypatch.setattr(C, "csa2_verify_drafts_workspace_bytes", lambda B, V: need[V])
    outs = []
    for V in (40, 400, 40):
        outs.append(step.verify(torch.zeros((5, V)), i(5), i(3), torch.zeros(5), torch.zeros(2)))
    gc.collect()
    assert len(made) == 2 and all(w() is not None for w in made)
    assert fake.calls[0][1][-2] == 512 and fake.calls[1][1][-2] == 4096
    assert outs[0][0] is outs[1][0] and outs[0][1] is outs[2][1]
    flags = []
    monkeypatch.setattr(C, "device_status", lambda ws, stream=None: flags.append(ws.data_ptr()) or 0)
    step.device_flags()
    assert {w().data_ptr() for w in made} <= set(flags)


# ---------------------------------------------------------------------------
# the plain forms themselves
# ---------------------------------------------------------------------------

def test_plain_verify_draws_from_the_target():
    """The emitted token's distribution is the target's, whatever the draft's (4 sigma of 40000 draws)."""
    rng = np.random.default_rng(3)
    p, q = np.array([.5, .25, .125, .125]), np.array([.1, .2, .3, .4])
    n = 40000
    x = rng.choice(4, n, p=q)
    tokens = np.stack([np.zeros(n, int), x], 1).reshape(-1)
    q_off = np.arange(n + 1) * 2
    tgt, drf = np.tile(p, (2 * n, 1)), np.tile(q, (2 * n, 1))
    a, t = R.verify(tgt, drf, tokens, q_off, rng.random(2 * n), rng.random(n))
    first = np.where(a == 1, x, t)
    freq = np.bincount(first, minlength=4) / n
    assert np.all(np.abs(freq - p) <= 4 * np.sqrt(p * (1 - p) / n))
    assert abs(a.mean() - np.minimum(p, q).sum()) <= 4 * 0.5 / np.sqrt(n)


def test_plain_evict_ranks():
    acc = np.array([0, 5, np.nan, 0, 7, -1, 0, 5], np.float32)
    assert list(R.evict_positions(acc, 3, 0, 0)) == [1, 4, 7]
    assert list(R.evict_positions(acc, 4, 1, 0)) == [0, 1, 4, 7]
    assert list(R.evict_positions(acc, 5, 0, 2)) == [0, 1, 4, 6, 7]
    assert list(R.evict_positions(acc, 7, 0, 0)) == [0, 1, 3, 4, 5, 6, 7]
    assert list(R.evict_positions(acc, 2, 3, 1)) == [0, 7]
    assert list(R.evict_positions(acc, -4, 1, 1)) == [] and list(R.evict_positions(acc, 99, 0, 0)) == list(range(8))


def test_dequant_matches_the_oracle():
    import oracle

    rng = np.random.default_rng(1)
    codes, scales = rng.integers(0, 256, (5, 256), dtype=np.uint8), rng.integers(100, 150, (5, 16), dtype=np.uint8)
    want = oracle.mxfp4_decode(codes, scales)
    assert np.array_equal(R.dequant(codes, scales), want.astype(np.float64))
