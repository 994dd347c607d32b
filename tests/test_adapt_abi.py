"""Host-side validation of the entry points around an adapted layer, and their
workspace queries (runs without a GPU: every call is refused before anything
is enqueued)."""

import ctypes
import os

import pytest

from int8_quantized_matmul_amd import _native

P, Q, R, U, V = (ctypes.c_void_p((1 << 20) + (k << 12)) for k in range(5))   # aligned stand-ins, never dereferenced
MIS2, MIS1 = ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 1)
F16, BF16, F32 = 0, 1, 2


def _lib():
    if not os.path.exists(_native.LIB_PATH):
        from int8_quantized_matmul_amd.build import build
        build()
    return _native.load()


def _norm(X=P, ldx=64, xt=F16, s=4, h=64, w=R, b=R, wt=F16, eps=1e-5, Y=Q, ldy=64, mean=U, rstd=V):
    return _lib().i8mm_layer_norm(X, ldx, xt, s, h, w, b, wt, eps, Y, ldy, mean, rstd, None)


def _norm_bwd(dY=P, lddy=64, X=Q, ldx=64, xt=F16, s=4, h=64, w=R, wt=F16, mean=U, rstd=V, dX=ctypes.c_void_p(1 << 30),
              lddx=64, dw=R, db=R, ws=P):
    return _lib().i8mm_layer_norm_backward(dY, lddy, X, ldx, xt, s, h, w, wt, mean, rstd, dX, lddx, dw, db, ws, None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(w=None), dict(Y=None), dict(xt=3), dict(xt=-1), dict(wt=BF16), dict(xt=F32, wt=F16),
    dict(s=-1), dict(s=1 << 31), dict(h=0), dict(h=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21), dict(ldx=63),
    dict(ldy=0), dict(ldx=-64), dict(ldx=1 << 40), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(X=MIS1), dict(Y=MIS1), dict(w=MIS1), dict(b=MIS1), dict(mean=MIS2), dict(rstd=MIS2), dict(wt=F32, w=MIS2),
    dict(xt=F32, wt=F32, X=MIS2), dict(Y=P, ldy=72)])
def test_layer_norm_rejects(kw):
    assert _norm(**kw) == -1


@pytest.mark.parametrize("kw", [
    dict(dY=None), dict(X=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dX=None), dict(ws=None),
    dict(ws=ctypes.c_void_p((1 << 20) + 128)), dict(dX=P), dict(dX=Q), dict(lddy=8), dict(lddx=63), dict(xt=5),
    dict(wt=BF16), dict(h=0), dict(s=-3), dict(dw=MIS2), dict(db=MIS2), dict(dX=MIS1)])
def test_layer_norm_backward_rejects(kw):
    assert _norm_bwd(**kw) == -1


def test_norm_workspace():
    q = _lib().i8mm_layer_norm_backward_workspace_bytes
    for s in (0, 1, 7, 4096, (1 << 31) - 1):
        for h in (1, 64, 12289, 1 << 20):
            assert q(s, h) >= 8 * h and q(s, h) % 256 == 0
    for s, h in ((-1, 64), (1 << 31, 64), (4, 0), (4, -1), (4, (1 << 20) + 1), (1 << 62, 1 << 62)):
        assert q(s, h) == 0


def _lora(X=P, ldx=128, A=R, B=R, t=F16, G=2, r=4, ids=U, scale=U, base=Q, ldb=64, s=4, h=128, o=64,
          Y=V, ldy=64, T=U, ws=P):
    return _lib().i8mm_lora_forward(X, ldx, A, B, t, G, r, ids, scale, base, ldb, s, h, o, Y, ldy, T, ws, None)


def _lora_bwd(dY=P, lddy=64, X=Q, ldx=128, T=U, A=R, B=R, t=F16, G=2, r=4, ids=U, scale=U, base=R, ldb=128, s=4, h=128,
              o=64, dX=V, lddx=128, dA=U, dB=U, ws=P):
    return _lib().i8mm_lora_backward(dY, lddy, X, ldx, T, A, B, t, G, r, ids, scale, base, ldb, s, h, o, dX, lddx, dA,
                                     dB, ws, None)


BAD_DIMS = [dict(s=-1), dict(s=16777217), dict(h=0), dict(h=96, ldx=96), dict(o=32), dict(o=65), dict(r=0), dict(r=129),
            dict(G=0), dict(G=65536), dict(h=133184, ldx=133184), dict(t=F32), dict(t=3), dict(ldx=120), dict(ldx=132),
            dict(ldb=60), dict(A=None), dict(B=None), dict(scale=None), dict(ids=None), dict(X=None), dict(ws=None),
            dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(A=ctypes.c_void_p((1 << 20) + 8)), dict(B=MIS2),
            dict(X=MIS2), dict(ids=MIS2), dict(scale=MIS2), dict(T=MIS2)]


@pytest.mark.parametrize("kw", BAD_DIMS + [dict(Y=None), dict(Y=P), dict(Y=Q, ldy=72), dict(ldy=68), dict(base=MIS2),
                                           dict(Y=MIS2)])
def test_lora_forward_rejects(kw):
    assert _lora(**kw) == -1


@pytest.mark.parametrize("kw", BAD_DIMS + [dict(dY=None), dict(T=None), dict(dA=None), dict(dB=None), dict(dX=P),
                                           dict(dX=Q), dict(dX=R, lddx=136), dict(lddx=130), dict(lddy=68),
                                           dict(dA=ctypes.c_void_p((1 << 20) + 4)), dict(dX=MIS2), dict(base=MIS2)])
def test_lora_backward_rejects(kw):
    assert _lora_bwd(**kw) == -1


def test_lora_workspaces():
    f, b = _lib().i8mm_lora_forward_workspace_bytes, _lib().i8mm_lora_backward_workspace_bytes
    for s, h, o, r in ((0, 64, 64, 1), (1, 64, 133120, 128), (16777216, 133120, 133120, 128), (4096, 12288, 36864, 16)):
        assert f(s, h, o, r) >= 4 * s * r
        for G in (1, 65535):
            assert b(s, h, o, r, G) >= 4 * s * r
    for s, h, o, r, G in ((-1, 64, 64, 1, 1), (1, 63, 64, 1, 1), (1, 64, 0, 1, 1), (1, 64, 64, 0, 1), (1, 64, 64, 129, 1),
                          (1, 64, 64, 1, 0), (1 << 62, 64, 64, 1, 1), (1, 64, 1 << 62, 1, 1)):
        assert b(s, h, o, r, G) == 0
        if G:
            assert f(s, h, o, r) == 0


def _clip(ptrs, numels, types, n=None, max_norm=1.0, outs=None, ws=P, total=Q):
    k = len(ptrs)
    arr = (ctypes.c_void_p * k)(*ptrs)
    out = None if outs is None else (ctypes.c_void_p * k)(*outs)
    return _lib().i8mm_clip_grad_norm(arr, out, (ctypes.c_int64 * k)(*numels), (ctypes.c_int32 * k)(*types),
                                      k if n is None else n, max_norm, ws, total, None)


def test_clip_rejects():
    a = 1 << 20
    assert _clip([a], [4], [F32], max_norm=-1.0) == -1
    assert _clip([a], [4], [F32], max_norm=float("nan")) == -1
    assert _clip([a], [4], [F32], ws=None) == -1
    assert _clip([a], [4], [F32], total=None) == -1
    assert _clip([a], [4], [F32], ws=ctypes.c_void_p(a + 64)) == -1
    assert _clip([a], [4], [F32], total=MIS2) == -1
    assert _clip([a], [4], [7]) == -1
    assert _clip([a], [-1], [F32]) == -1
    assert _clip([a], [1 << 60], [F32]) == -1
    assert _clip([a, a], [1 << 46, 1 << 46], [F32, F32]) == -1
    assert _clip([a + 2], [4], [F32]) == -1
    assert _clip([a + 1], [4], [BF16]) == -1
    assert _clip([None], [4], [F32]) == -1
    assert _clip([a], [4], [F32], outs=[None]) == -1
    assert _clip([a], [4], [F32], outs=[a + 2]) == -1
    assert _clip([a], [4], [F32], n=-1) == -1
    lib = _lib()
    assert lib.i8mm_clip_grad_norm(None, None, None, None, 2, 1.0, P, Q, None) == -1


def test_clip_workspace():
    q = _lib().i8mm_clip_grad_norm_workspace_bytes
    assert q(None, 0) >= 256 and q(None, 1) == 0 and q(None, -1) == 0
    n = (ctypes.c_int64 * 3)(0, 5, 10 ** 9)
    assert q(n, 3) >= q(n, 2) >= 256
    assert q((ctypes.c_int64 * 2)(1, -1), 2) == 0


def test_valid_calls_without_gpu_report_no_device():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert _norm() == -2 and _norm_bwd() == -2 and _lora() == -2 and _lora_bwd() == -2
    assert _norm(s=0, X=None, Y=None) == -2 and _lora(s=0, X=None, ids=None, Y=None) == -2
    assert _norm(Y=P) == -2 and _lora(Y=Q) == -2
    assert _clip([1 << 20], [4], [F32]) == -2 and _clip([], [], []) == -2
