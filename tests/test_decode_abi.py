"""Host-side validation of the entry points of decoding (paged cache, its
attention, beam selection) and their workspace queries (runs without a GPU:
every call is refused before anything is enqueued)."""

import ctypes
import os

import pytest

from int8_quantized_matmul_amd import _native

P, Q, R, U, V, W, X, Y = (ctypes.c_void_p((1 << 20) + (k << 12)) for k in range(8))   # aligned, never dereferenced
MIS8, MIS2, MIS64 = (ctypes.c_void_p((1 << 20) + k) for k in (8, 2, 64))
F16, BF16, F32 = 0, 1, 2
BIG = [-1, -(1 << 63), (1 << 63) - 1, 1 << 62, 1 << 41]


def _lib():
    if not os.path.exists(_native.LIB_PATH):
        from int8_quantized_matmul_amd.build import build
        build()
    return _native.load()


def _append(K=P, ldk=128, Vr=Q, ldv=128, t=F16, s=4, kv=2, d=64, seq=R, pos=U, tables=V, ldt=8, n=4, M=8, Kp=W, ks=2048, Vp=X,
            vs=2048, pages=9, page=16):
    return _lib().i8mm_cache_append(K, ldk, Vr, ldv, t, s, kv, d, seq, pos, tables, ldt, n, M, Kp, ks, Vp, vs, pages, page, None)


BAD_CACHE = [dict(kv=0), dict(d=0), dict(d=12), dict(d=264, ldk=1 << 12, ldv=1 << 12, ks=1 << 20, vs=1 << 20), dict(page=8),
             dict(page=24), dict(page=0), dict(page=-16), dict(page=4112), dict(pages=0), dict(pages=(1 << 24) + 1), dict(M=0),
             dict(M=(1 << 20) + 1, ldt=1 << 30), dict(M=1 << 20, ldt=1 << 30, page=4096, ks=1 << 30, vs=1 << 30), dict(ldt=7),
             dict(n=-1), dict(n=(1 << 20) + 1), dict(t=F32), dict(t=-1), dict(t=3), dict(ks=2047), dict(vs=2040),
             dict(ks=2052), dict(vs=1 << 41), dict(tables=None), dict(tables=MIS2)]


@pytest.mark.parametrize("kw", BAD_CACHE + [dict(K=None), dict(Vr=None), dict(pos=None), dict(Kp=None), dict(Vp=None),
                                            dict(K=MIS8), dict(Vr=MIS2), dict(Kp=MIS8), dict(Vp=MIS2), dict(seq=MIS2),
                                            dict(pos=MIS2), dict(ldk=120), dict(ldv=132), dict(s=-1), dict(s=(1 << 24) + 1)])
def test_append_rejects(kw):
    assert _append(**kw) == -1


@pytest.mark.parametrize("name", ["ldk", "ldv", "s", "kv", "d", "ldt", "n", "M", "ks", "vs", "pages", "page"])
def test_append_rejects_extremes(name):
    assert all(_append(**{name: v}) == -1 for v in BIG)


def _attend(q=P, ldq=256, t=F16, n=4, heads=4, kv=2, d=64, Kp=W, ks=2048, Vp=X, vs=2048, pages=9, page=16, tables=V, ldt=8, M=8,
            lens=R, beams=2, scale=0.1, slopes=U, out=Y, ldo=256, lse=Q, ws=P):
    return _lib().i8mm_decode_attention(q, ldq, t, n, heads, kv, d, Kp, ks, Vp, vs, pages, page, tables, ldt, M, lens, beams,
                                        scale, slopes, out, ldo, lse, ws, None)


@pytest.mark.parametrize("kw", [{("ldq" if k == "ldk" else "ldo" if k == "ldv" else k): v for k, v in kw.items()}
                                for kw in BAD_CACHE]
                         + [dict(q=None), dict(out=None), dict(lens=None), dict(Kp=None), dict(Vp=None), dict(ws=None, M=33, ldt=33), dict(ws=None, M=65, ldt=65, beams=1),
                            dict(ws=MIS64), dict(q=MIS8), dict(out=MIS2), dict(out=P), dict(lens=MIS2), dict(slopes=MIS2),
                            dict(lse=MIS2), dict(heads=3), dict(heads=1), dict(heads=65536), dict(heads=0), dict(beams=0),
                            dict(beams=3), dict(beams=65, n=65), dict(scale=float("nan")), dict(scale=float("inf")),
                            dict(ldq=248), dict(ldo=260), dict(Kp=MIS8), dict(Vp=MIS2)])
def test_attention_rejects(kw):
    assert _attend(**kw) == -1


@pytest.mark.parametrize("name", ["ldq", "ldo", "n", "heads", "kv", "d", "ldt", "M", "ks", "vs", "pages", "page", "beams"])
def test_attention_rejects_extremes(name):
    assert all(_attend(**{name: v}) == -1 for v in BIG)


def _host(values, kind=ctypes.c_int64):
    return None if values is None else (kind * max(1, len(values)))(*values)


def _fork(tables=P, ldt=8, lens=Q, refs=R, n=4, M=8, pages=9, page=16, parents=U, grow=U, m=5, to=V, ldto=8, lo=W, ro=X, state=Y,
          at=(1 << 20,), size=(4096,), step=(4096,), pools=None, ws=P):
    return _lib().i8mm_cache_fork(tables, ldt, lens, refs, n, M, pages, page, parents, grow, m, to, ldto, lo, ro, state,
                                  _host(at, ctypes.c_void_p), _host(size), _host(step), len(at or ()) if pools is None else pools,
                                  ws, None)


BAD_POOLS = [dict(pools=-1), dict(pools=65537), dict(at=(None,)), dict(at=((1 << 20) + 8,)), dict(size=(0,)), dict(size=(24,)),
             dict(size=(-16,)), dict(size=((1 << 32) + 16,), step=(1 << 33,)), dict(step=(4080,)), dict(step=(4104,)),
             dict(step=(1 << 41,)), dict(at=None, pools=1), dict(size=None), dict(step=None)]


@pytest.mark.parametrize("kw", BAD_POOLS + [
    dict(tables=None), dict(lens=None), dict(refs=None), dict(to=None), dict(lo=None), dict(ro=None), dict(state=None),
    dict(ws=None), dict(ws=MIS64), dict(tables=MIS2), dict(lens=MIS2), dict(refs=MIS2), dict(parents=MIS2), dict(grow=MIS2),
    dict(to=MIS2), dict(lo=MIS2), dict(ro=MIS2), dict(state=MIS2), dict(to=P), dict(lo=Q), dict(ro=R), dict(ldt=7), dict(ldto=7),
    dict(page=8), dict(page=20), dict(pages=0), dict(M=0), dict(n=-1), dict(m=-1), dict(m=(1 << 20) + 1)])
def test_fork_rejects(kw):
    assert _fork(**kw) == -1


@pytest.mark.parametrize("name", ["ldt", "n", "M", "pages", "page", "m", "ldto"])
def test_fork_rejects_extremes(name):
    assert all(_fork(**{name: v}) == -1 for v in BIG)


def _compact(tables=P, ldt=8, n=4, M=8, refs=R, pages=9, to=V, ldto=8, ro=X, moved=U, state=Y, at=(1 << 20,), size=(4096,),
             step=(4096,), pools=None, ws=P):
    return _lib().i8mm_cache_compact(tables, ldt, n, M, refs, pages, to, ldto, ro, moved, state, _host(at, ctypes.c_void_p),
                                     _host(size), _host(step), len(at or ()) if pools is None else pools, ws, None)


@pytest.mark.parametrize("kw", BAD_POOLS + [
    dict(tables=None), dict(refs=None), dict(to=None), dict(ro=None), dict(moved=None), dict(state=None), dict(ws=None),
    dict(ws=MIS64), dict(tables=MIS2), dict(refs=MIS2), dict(to=MIS2), dict(ro=MIS2), dict(moved=MIS2), dict(state=MIS2),
    dict(ro=R), dict(to=P, ldto=9), dict(ldt=7), dict(ldto=7), dict(pages=0), dict(M=0), dict(n=-1)])
def test_compact_rejects(kw):
    assert _compact(**kw) == -1


@pytest.mark.parametrize("name", ["ldt", "n", "M", "pages", "ldto"])
def test_compact_rejects_extremes(name):
    assert all(_compact(**{name: v}) == -1 for v in BIG)


def _select(x=P, ld=100, t=F16, n=3, beams=4, vocab=100, scores=Q, k=8, so=R, parents=U, tokens=V, h=W, ldh=7, T=7, ho=X, ldho=8,
            ws=P):
    return _lib().i8mm_beam_select(x, ld, t, n, beams, vocab, scores, k, so, parents, tokens, h, ldh, T, ho, ldho, ws, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(scores=None), dict(so=None), dict(parents=None), dict(tokens=None), dict(ws=None), dict(ws=MIS64),
    dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(t=F32, x=MIS2), dict(scores=MIS2), dict(so=MIS2), dict(parents=MIS2),
    dict(tokens=MIS2), dict(so=Q), dict(t=3), dict(t=-1), dict(ld=99), dict(beams=0), dict(beams=65), dict(k=0), dict(k=65),
    dict(beams=1, vocab=7, k=8), dict(vocab=0), dict(vocab=(1 << 24) + 1, ld=1 << 30), dict(n=-1), dict(n=(1 << 20) + 1),
    dict(h=None), dict(h=X), dict(ldh=6), dict(ldho=7), dict(T=-1), dict(h=MIS2), dict(ho=MIS2)])
def test_select_rejects(kw):
    assert _select(**kw) == -1


@pytest.mark.parametrize("name", ["ld", "n", "beams", "vocab", "k", "ldh", "T", "ldho"])
def test_select_rejects_extremes(name):
    assert all(_select(**{name: v}) == -1 for v in BIG)


def test_workspaces():
    lib = _lib()
    fork, compact, attend, select = (lib.i8mm_cache_fork_workspace_bytes, lib.i8mm_cache_compact_workspace_bytes,
                                     lib.i8mm_decode_attention_workspace_bytes, lib.i8mm_beam_select_workspace_bytes)
    for n, m, pages in ((0, 0, 1), (1, 1, 1), (1 << 20, 1 << 20, 1 << 24), (7, 300, 12345)):
        assert 0 < fork(n, m, pages) < 2 ** 29 and fork(n, m, pages) % 256 == 0
    for args in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1 << 21, 1, 1), (1, 1, 1 << 25)):
        assert fork(*args) == 0
    assert 4 <= compact(1) < compact(1 << 24) < 2 ** 29 and compact(0) == compact((1 << 24) + 1) == compact(-1) == 0
    for n, heads, kv, d in ((0, 1, 1, 8), (1, 1, 1, 128), (64, 96, 96, 128), (1 << 20, 65535, 1, 256), (32, 64, 8, 80)):
        assert 0 < attend(n, heads, kv, d) < 2 ** 30 and attend(n, heads, kv, d) % 256 == 0
    for args in ((-1, 4, 4, 64), (1, 5, 4, 64), (1, 0, 0, 64), (1, 4, 4, 60), (1, 4, 4, 264), (1, 65536, 1, 64), (1, 4, 8, 64)):
        assert attend(*args) == 0
    for n, beams, vocab, k in ((0, 1, 1, 1), (1, 64, 1, 64), (64, 8, 50257, 16), (1 << 20, 64, 1 << 24, 64)):
        assert select(n, beams, vocab, k) >= 256 and select(n, beams, vocab, k) % 256 == 0
    for args in ((1, 65, 8, 8), (1, 1, 0, 1), (1, 2, 3, 7), (-1, 1, 1, 1), (1, 1, 1 << 25, 1), (1 << 62, 1, 1, 1)):
        assert select(*args) == 0


def test_valid_calls_without_gpu_report_no_device():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert _append() == _attend() == _fork() == _compact() == _select() == -2
    assert _append(seq=None) == -2 and _append(s=0, K=None, Vr=None, pos=None) == -2 and _append(n=0, tables=None) == -2
    assert _attend(slopes=None, lse=None) == -2 and _attend(ws=None, M=32, ldt=32) == _attend(ws=None, M=64, ldt=64, beams=1) == -2 and _attend(n=0, q=None, out=None, lens=None, tables=None) == -2
    assert _fork(parents=None, grow=None, at=(), size=(), step=()) == -2 and _fork(n=0, tables=None, lens=None) == -2
    assert _fork(m=0, to=None, lo=None) == -2 and _compact(to=P) == -2 and _compact(n=0, tables=None, to=None) == -2
    assert _select(ho=None, h=None, T=-5) == -2 and _select(h=None, T=0) == -2 and _select(t=F32) == -2
