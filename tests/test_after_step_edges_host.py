"""Edges of the calls that follow a step, without a GPU: what they refuse, and
how the step's orchestration keeps the layers' caches in step."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from long_context_decode_csa2_b200 import _build
from long_context_decode_csa2_b200 import csa2 as C
from long_context_decode_csa2_b200.decode import DecodeStep, FullCache, PairStream, clear_acc, evict
from tests.test_binding_host import fake  # noqa: F401  (fixture)

GIB = 1 << 30


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def _z(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _full_cache(rows=64, acc=True):
    return FullCache(C.cache(_z(rows, 64), _z(rows, 4)), C.cache(_z(rows, 256), _z(rows, 16)),
                     torch.zeros(rows) if acc else None)


# ---------------------------------------------------------------------------
# eviction of several layers
# ---------------------------------------------------------------------------

def _layers(n=2, paged=False, dst=lambda i, plane: (8 + i) * GIB + (plane << 26), src=lambda i, plane: (1 + i) * GIB + (plane << 26),
            acc_src=None, acc_dst=None, idx=True, rows=1024, B=2, idx_dst=True, page_rows=512):
    caches = lambda at, a, b: (C.MXFP4Cache * max(n, 1))(*(C.MXFP4Cache(at(i, a), at(i, b), rows) for i in range(n)))  # noqa: E731
    ptrs = lambda v, at: (ctypes.c_void_p * max(n, 1))(*(v or [at(i, 4) for i in range(n)]))  # noqa: E731
    ms, md, xs, xd = caches(src, 0, 1), caches(dst, 0, 1), caches(src, 2, 3), caches(dst, 2, 3)
    head = [n, ms, xs if idx else None, ptrs(acc_src, src)]
    there = [md, xd if idx and idx_dst else None, ptrs(acc_dst, dst)]
    tail = [GIB >> 1, GIB >> 1, B, 512, 256, 0, 0, GIB >> 1, 255, None]   # the workspace is one byte short
    fake_at = GIB >> 1
    if paged:
        return C.lib().csa2_cache_evict_layers_paged(*head, fake_at, 4, fake_at, fake_at, *there, fake_at, 4, page_rows, *tail)
    return C.lib().csa2_cache_evict_layers(*head, fake_at, fake_at, fake_at, *there, fake_at, *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_evict_layers_refuses(paged):
    """A call that is sound but for its workspace answers -3; what is wrong is refused before that, or with it."""
    call = lambda **kw: _layers(paged=paged, **kw)  # noqa: E731
    assert call() == -3 and call(n=1) == -3 and call(n=64) == -3 and call(idx=False) == -3
    assert call(n=0) == -2 and call(n=65) == -2 and call(n=-1) == -2 and call(idx_dst=False) == -1
    assert call(B=0) == 0 and call(B=-1) == -1 and call(rows=1001) == -1
    if paged:
        assert call(page_rows=500) == -1


@pytest.mark.parametrize("paged", [False, True])
def test_evict_layers_refuses_memory_of_two_layers(paged, monkeypatch):
    """Overlaps are looked for once everything else is sound: with a workspace, and none of these calls launches."""
    src, dst = (lambda i, plane: (1 + i) * GIB + (plane << 26)), (lambda i, plane: (8 + i) * GIB + (plane << 26))

    def call(ws_bytes=256, **kw):
        L = C.lib()
        name = "csa2_cache_evict_layers" + ("_paged" if paged else "")
        real = getattr(L, name)
        with monkeypatch.context() as m:
            m.setattr(L, name, lambda *a: real(*a[:-2], ws_bytes, a[-1]))
            return _layers(paged=paged, **kw)

    assert call(dst=lambda i, plane: 8 * GIB + (plane << 26)) == -1                    # one destination for both
    assert call(dst=lambda i, plane: src(1 - i, plane)) == -1                          # each other's source
    assert call(dst=lambda i, plane: dst(i, plane) if plane != 3 else dst(0, 3)) == -1  # indexer scales alone
    assert call(acc_dst=[dst(0, 4)] * 2) == -1                                         # two layers' weights to one place
    assert call(acc_src=[src(0, 4)] * 2, acc_dst=[dst(0, 4), dst(0, 4) + 8]) == -1
    assert call(acc_dst=[src(1, 4), dst(1, 4)]) == -1
    if not paged:
        assert call(dst=src) == -1
        assert call(acc_src=[src(0, 4)] * 2, acc_dst=[src(0, 4)] * 2) == -1
    assert b"overlap" in C.lib().csa2_last_error()


def _evict_args(n):
    off = torch.zeros(2, dtype=torch.int64)
    return dict(src_rows=off, dst_rows=off, seq_len=_i(2), keep=_i(2), max_len=32, max_keep=16, kept=_i(2, 16),
                seq_len_out=_i(2), ws=_z(256))


def test_evict_of_a_steps_layers(fake):  # noqa: F811
    """Full layers that select in the first one's pool are evicted together; a lone one of them is refused."""
    args = _evict_args(2)
    src, dst = [_full_cache() for _ in range(2)], [_full_cache() for _ in range(2)]
    evict(src[0], dst[0], **args)                        # nothing says that it has company: a cache of its own
    step = DecodeStep("FUFR", 2, 32, 16, 8, device="cpu", concurrent=False)
    layers = [dict(q=torch.zeros((2, 16, 512), dtype=torch.bfloat16)) for _ in range(4)]
    step.accumulate(src, args["src_rows"], args["seq_len"], layers)
    fake.calls.clear()
    for lone in (src[0], [src[1]]):
        with pytest.raises(ValueError, match="2 Full layers"):
            evict(lone, dst[0], **args)
    assert not fake.calls
    evict(src, dst, **args)
    (name, a), = fake.calls
    assert name == "csa2_cache_evict_layers" and a[0] == 2
    for f in range(2):
        assert a[1][f].codes == src[f].main.codes and a[2][f].scales == src[f].idx.scales
        assert a[3][f] == src[f].acc.data_ptr() and a[9][f] == dst[f].acc.data_ptr()
        assert a[7][f].scales == dst[f].main.scales and a[8][f].codes == dst[f].idx.codes
    with pytest.raises(ValueError, match="2 Full layers"):
        evict(dst[1], src[1], **args)                    # what was evicted together goes on together
    pt = C.PageTable(_i(2, 1), 512)
    evict(src, dst, **{**args, "src_rows": pt, "dst_rows": pt})
    assert fake.calls[-1][0] == "csa2_cache_evict_layers_paged"
    with pytest.raises(ValueError, match="as many"):
        evict(src, dst[:1], **args)
    with pytest.raises(ValueError, match="at least one"):
        evict([], [], **args)
    with pytest.raises(ValueError, match="acc"):
        evict(src, [dst[0], _full_cache(acc=False)], **args)
    # layers that scan for themselves keep what they like
    DecodeStep("FUFR", 2, 32, 16, 8, device="cpu", concurrent=False, full_rescan=True).accumulate(
        src, args["src_rows"], args["seq_len"], layers)
    evict(src[1], dst[1], **args)
    assert fake.calls[-1][0] == "csa2_cache_evict"


def test_evict_layers_binding_checks(fake):  # noqa: F811
    src, dst = [_full_cache() for _ in range(2)], [_full_cache() for _ in range(2)]
    off = torch.zeros(2, dtype=torch.int64)
    pt = C.PageTable(_i(2, 1), 512)
    base = dict(main_src=[c.main for c in src], idx_src=[c.idx for c in src], acc_src=[c.acc for c in src], src=off,
                seq_len=_i(2), keep=_i(2), max_len=32, max_keep=16, main_dst=[c.main for c in dst],
                idx_dst=[c.idx for c in dst], acc_dst=[c.acc for c in dst], dst=off, kept=_i(2, 16), seq_len_out=_i(2),
                ws=_z(256))
    for change in (dict(src=pt), dict(dst=pt), dict(src=pt, dst=C.PageTable(_i(2, 1), 1024)), dict(idx_dst=None),
                   dict(main_src=[src[0].main]), dict(acc_dst=[dst[0].acc]), dict(kept=_i(2, 15)),
                   dict(acc_src=[src[0].acc, torch.zeros(63)]), dict(acc_dst=[dst[0].acc, torch.zeros(64).double()]),
                   dict(main_src=[], idx_src=[], acc_src=[], main_dst=[], idx_dst=[], acc_dst=[])):
        with pytest.raises(C.Csa2Error):
            C.csa2_cache_evict_layers(**{**base, **change})
    assert not fake.calls
    C.csa2_cache_evict_layers(**{**base, "idx_src": None, "idx_dst": None})
    (_, a), = fake.calls
    assert a[2][0].codes is None and a[8][1].codes is None


# ---------------------------------------------------------------------------
# accumulators of new entries
# ---------------------------------------------------------------------------

def test_acc_clear_refuses():
    L, at = C.lib(), GIB

    def call(acc=at, rows=1024, off=at, a=at, b=at, B=2, ws=at, wn=256):
        return L.csa2_acc_clear(acc, rows, off, a, b, B, ws, wn, None)

    def paged(rows=1024, pages=at, page_rows=512, max_pages=2, B=2, wn=255):
        return L.csa2_acc_clear_paged(at, rows, pages, page_rows, max_pages, at, at, B, at, wn, None)

    assert call(wn=255) == -3 and paged() == -3
    for bad in (dict(acc=None), dict(off=None), dict(a=None), dict(b=None), dict(ws=None), dict(ws=at + 8), dict(B=-1),
                dict(rows=-8)):
        assert call(**{"wn": 255, **bad}) == -1
    for bad in (dict(rows=1000), dict(pages=None), dict(page_rows=300), dict(max_pages=0), dict(B=-1)):
        assert paged(**bad) == -1
    assert call(B=0) == 0 and paged(B=0) == 0


def test_ratio2_appends_start_accumulators_at_zero(fake):  # noqa: F811
    """Behind every append the new entries' accumulators are cleared, with the lengths before and after it; caches
    without accumulators append as ever."""
    off, lens = torch.zeros(2, dtype=torch.int64), torch.tensor([3, 5], dtype=torch.int32)
    tok = dict(raw=torch.zeros((2, 512), dtype=torch.bfloat16), logit=torch.zeros(2), w_idx=torch.zeros((512, 128)))
    pair = PairStream(2, "cpu")
    for with_acc in (False, True):
        for update in (False, True):
            cache = _full_cache(acc=with_acc)
            lens.copy_(torch.tensor([3, 5], dtype=torch.int32))
            pair.new_len.copy_(torch.tensor([4, 5], dtype=torch.int32))     # as the library would leave it
            fake.calls.clear()
            pair.append(cache, tok, off, lens, update)
            (name, a), *rest = fake.calls
            out = pair.new_len.data_ptr() if with_acc else lens.data_ptr() if update else None
            assert name == "csa2_compress_stream" and a[8] == lens.data_ptr() and a[9] == out
            assert [n for n, _ in rest] == ["csa2_acc_clear"] * with_acc
            if with_acc:
                (_, c), = rest
                assert c[0] == cache.acc.data_ptr() and c[1] == 64 and c[3:5] == (lens.data_ptr(), out)
            assert lens.tolist() == ([4, 5] if with_acc and update else [3, 5])
    fake.calls.clear()
    clear_acc([_full_cache(), _full_cache(acc=False)], C.PageTable(_i(2, 1), 512), _i(2), lens, _z(256))
    assert [n for n, _ in fake.calls] == ["csa2_acc_clear_paged"]
    for bad in (dict(acc=torch.zeros(63)), dict(len_from=_i(1)), dict(len_to=torch.zeros(2))):
        args = dict(acc=torch.zeros(64), seq_row_off=off, len_from=_i(2), len_to=lens, ws=_z(256), rows=64)
        with pytest.raises(C.Csa2Error):
            C.csa2_acc_clear(**{**args, **bad})


# ---------------------------------------------------------------------------
# launches from several threads
# ---------------------------------------------------------------------------

_RUNTIME = r"""
// The runtime calls of a launch, recorded: a kernel's dynamic shared memory limit and what launches ask of it.
#include <cuda_runtime_api.h>
#include <stdio.h>
#define API extern "C" __attribute__((visibility("default")))
API cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) printf("limit %p %d\n", f, value);
  return cudaSuccess;
}
API cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  printf("launch %p %zu\n", f, c->dynamicSmemBytes);
  return cudaSuccess;
}
API cudaError_t cudaGetLastError(void) { return cudaSuccess; }
"""

_EVICT_OF_ALL_SIZES = """
import sys
from long_context_decode_csa2_b200 import _build
from long_context_decode_csa2_b200 import csa2 as C
import ctypes
import os
import subprocess
import sys
L, at, G = C.lib(), 1 << 29, 1 << 30
cache = lambda i: (C.MXFP4Cache * 3)(*(C.MXFP4Cache((i + l) * G, (i + l) * G + (1 << 29), 1 << 20) for l in range(3)))
for n_layers in (1, 3):
    for max_len in (0, 1000, 20000, 60000, 120000, 300000, 700000, 1 << 20, 1 << 24):
        for B in (1, 40):
            src, dst = cache(1), cache(8)
            acc = [(ctypes.c_void_p * 3)(*((i + l) * G + (3 << 28) for l in range(3))) for i in (20, 30)]
            rc = L.csa2_cache_evict_layers(n_layers, src, None, acc[0], at, at, at, dst, None, acc[1], at, at, at, B, max_len,
                                           64, 0, 0, at, 256, None)
            assert rc == 0, (rc, L.csa2_last_error())
"""


def test_evict_sets_one_shared_memory_limit_for_all_sizes(tmp_path):
    """The limit belongs to the kernel, not to the call: two threads that set their own sizes could launch under each
    other's.  Recorded with a stand-in of the runtime's launch calls: one value per kernel, and every launch within it."""
    src, lib = tmp_path / "runtime.cpp", tmp_path / "runtime.so"
    src.write_text(_RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", include, str(src), "-o", str(lib)], check=True)
    _build.build()
    r = subprocess.run([sys.executable, "-c", _EVICT_OF_ALL_SIZES], cwd=_build.ROOT, capture_output=True, text=True,
                       env={**os.environ, "LD_PRELOAD": str(lib)})
    assert r.returncode == 0, r.stderr
    said = [line.split() for line in r.stdout.splitlines()]
    limits = {}
    for what, f, value in said:
        if what == "limit":
            limits.setdefault(f, set()).add(int(value))
    sizes = [(f, int(v)) for what, f, v in said if what == "launch" and int(v) > 48 * 1024]
    assert len({v for _, v in sizes}) > 3 and len({f for f, _ in sizes}) == 2     # one layer, and several
    assert all(len(v) == 1 for v in limits.values()), limits
    assert all(v <= max(limits[f]) for f, v in sizes)


# ---------------------------------------------------------------------------
# outputs whose rows lie apart
# ---------------------------------------------------------------------------

def test_outputs_with_other_row_lengths_are_refused(fake):  # noqa: F811
    """The library writes rows of max_keep (or k) elements: in a wider buffer every row but the first would lie elsewhere
    than its index says.  A flat buffer holds the rows one behind the other."""
    src, dst = _full_cache(), _full_cache()
    off, ws = torch.zeros(2, dtype=torch.int64), _z(256)
    one = lambda kept: C.csa2_cache_evict(  # noqa: E731
        src.main, src.idx, src.acc, off, _i(2), _i(2), 32, 16, dst.main, dst.idx, dst.acc, off, kept, _i(2), ws)
    many = lambda kept: C.csa2_cache_evict_layers(  # noqa: E731
        [src.main] * 2, None, [src.acc] * 2, off, _i(2), _i(2), 32, 16, [dst.main] * 2, None, [dst.acc] * 2, off, kept,
        _i(2), ws)
    for call in (one, many):
        for bad in (_i(2, 17), _i(2, 20), _i(1, 32), _i(4, 8), _i(2, 1, 16), _i(31), [0] * 32):
            with pytest.raises(C.Csa2Error, match="kept"):
                call(bad)
        assert not fake.calls
        for good in (_i(2, 16), _i(3, 16), _i(32), _i(40)):
            call(good)
        assert len(fake.calls) == 4
        fake.calls.clear()
    weights = lambda w: C.csa2_attn_weights(  # noqa: E731
        torch.zeros((2, 16, 512), dtype=torch.bfloat16), src.main, off, _i(2), _i(2, 8), torch.zeros((2, 16)), 0.1, src.acc,
        ws, weights=w)
    for bad in (torch.zeros((2, 9)), torch.zeros((1, 16)), torch.zeros((4, 4)), torch.zeros(15)):
        with pytest.raises(C.Csa2Error, match="weights"):
            weights(bad)
    assert not fake.calls
    for good in (torch.zeros((2, 8)), torch.zeros((5, 8)), torch.zeros(16), None):
        weights(good)


# ---------------------------------------------------------------------------
# offsets near the end of 64 bits
# ---------------------------------------------------------------------------

def test_prefill_refuses_rows_whose_sum_wraps():
    """A row offset so large that its sum with the length is negative lies outside the cache like any other."""
    L, at, cache = C.lib(), GIB, C.MXFP4Cache(GIB, GIB, 4096)

    def index(row0, n=1024):
        return L.csa2_index_prefill(cache, at, at, at, at, 4, row0, n, 1, 64, 64, at, at, at, 255, None)

    def attend(row0, n=1024):
        return L.csa2_sparse_attn_prefill(at, at, 4, cache, row0, n, 1, at, 64, at, 100, 1.0, 0.1, at, None, at, 255, None)

    for call in (index, attend):
        assert call(0) == call(3072) == -3                  # sound but for the workspace
        for row0 in (3080, 2 ** 31 - 8, 2 ** 63 - 8, 2 ** 63 - 1024):
            assert call(row0) == -1
        assert call(0, 2 ** 31) == -1 and call(0, 4104) == -1


def test_verification_steps_take_row_offsets(fake):  # noqa: F811
    step = DecodeStep("FU", 2, 32, 16, 8, device="cpu", concurrent=False, queries=5)
    with pytest.raises(ValueError, match="row offsets"):
        step.run([_full_cache()], C.PageTable(_i(2, 1), 512), _i(2), [{}, {}], q_off=_i(3), q_vis=_i(5))
    assert not fake.calls
