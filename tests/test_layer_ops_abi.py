"""CPU: the state space layer's operators reject bad arguments on the host, before anything is
launched, and their fp64 definitions agree with closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_71_b200 as gdn
from gated_delta_rule_71_b200 import _lib
from oracle import layer

OK, INVALID, UNSUPPORTED = 0, 1, 2
p, q, big = ctypes.c_void_p(256), ctypes.c_void_p(512), 1 << 40


def scan(**kw):
    a = dict(x=p, xs=64 * 8, dt=p, dts=8, Bm=p, bs=2 * 64, Cm=p, cs=2 * 64, z=None, zs=0, ty=1, A=p,
             bias=p, D=None, h0=None, cu=None, n_seq=0, B=2, T=40, H=8, G=2, P=64, N=64, y=q, hT=None,
             ws=q, wsb=big)
    a.update(kw)
    return _lib.load().gdn_ssm_scan(
        a["x"], a["xs"], a["dt"], a["dts"], a["Bm"], a["bs"], a["Cm"], a["cs"], a["z"], a["zs"], a["ty"],
        a["A"], a["bias"], a["D"], a["h0"], a["cu"], a["n_seq"], a["B"], a["T"], a["H"], a["G"], a["P"],
        a["N"], a["y"], a["hT"], a["ws"], a["wsb"], None)


def test_scan_refusals():
    for bad in (dict(H=9), dict(G=0), dict(H=0), dict(B=-1), dict(T=-1), dict(ty=7), dict(xs=511),
                dict(dts=7), dict(bs=127), dict(cs=127), dict(z=p, zs=511), dict(x=None), dict(dt=None),
                dict(Bm=None), dict(Cm=None), dict(y=None), dict(A=None), dict(bias=None), dict(y=p),
                dict(z=q, zs=512), dict(x=ctypes.c_void_p(257)), dict(h0=ctypes.c_void_p(258)),
                dict(h0=q, hT=q), dict(cu=p, n_seq=2, B=2), dict(cu=p, n_seq=-1, B=1),
                dict(cu=ctypes.c_void_p(258), n_seq=2, B=1)):
        assert scan(**bad) == INVALID, bad
    for bad in (dict(P=96, xs=big), dict(N=16), dict(P=256, xs=big), dict(T=1 << 41)):
        assert scan(**bad) == UNSUPPORTED, bad
    assert scan(B=0) == OK
    assert scan(cu=p, n_seq=0, B=1) == OK


def test_scan_workspace():
    lib = _lib.load()
    need = lib.gdn_ssm_scan_workspace_size(2, 80, 8, 2, 64, 64, 1)
    if need:
        assert scan(ws=None) == INVALID
        assert scan(wsb=need - 1) == INVALID
        assert scan(ws=ctypes.c_void_p(520)) == INVALID
    assert lib.gdn_ssm_scan_workspace_size(0, 80, 8, 2, 64, 64, 1) == 0
    assert lib.gdn_ssm_scan_workspace_size(2, 80, 8, 0, 64, 64, 1) == 0
    assert lib.gdn_ssm_scan_workspace_size(2, 80, 8, 2, 64, 64, 0) == 0  # fp32: no workspace


def step(**kw):
    C = 8 * 64 + 4 * 64
    a = dict(row=p, rs=C, dt=p, dts=8, z=None, zs=0, w=p, cb=None, W=4, cst=p, act=1, A=p, bias=p,
             D=None, n=5, H=8, G=2, P=64, N=64, st=p, idx=None, slots=5, y=q, ws=p, wsb=big)
    a.update(kw)
    return _lib.load().gdn_ssm_decode_step(
        a["row"], a["rs"], a["dt"], a["dts"], a["z"], a["zs"], a["w"], a["cb"], a["W"], a["cst"],
        a["act"], a["A"], a["bias"], a["D"], a["n"], a["H"], a["G"], a["P"], a["N"], a["st"], a["idx"],
        a["slots"], a["y"], a["ws"], a["wsb"], None)


def test_step_refusals():
    need = _lib.load().gdn_ssm_decode_step_workspace_size(5, 8, 2, 64, 64)
    assert need >= 5 * (8 * 64 + 4 * 64) * 4
    for bad in (dict(n=-1), dict(H=9), dict(W=0), dict(W=5), dict(act=2), dict(rs=767), dict(dts=7),
                dict(z=p, zs=511), dict(row=None), dict(dt=None), dict(w=None), dict(cst=None),
                dict(A=None), dict(bias=None), dict(y=None), dict(y=p), dict(slots=-1), dict(slots=4),
                dict(st=None), dict(st=ctypes.c_void_p(264)), dict(idx=ctypes.c_void_p(258)),
                dict(ws=None), dict(wsb=need - 1), dict(ws=ctypes.c_void_p(264))):
        assert step(**bad) == INVALID, bad
    for bad in (dict(P=48, rs=big), dict(N=256, rs=big), dict(n=1 << 30, slots=1 << 30)):
        assert step(**bad) in (UNSUPPORTED, INVALID), bad
    assert step(n=0) == OK
    assert _lib.load().gdn_ssm_decode_step_workspace_size(0, 8, 2, 64, 64) == 0


def test_norm_refusals():
    f = _lib.load().gdn_rmsnorm_fp8

    def norm(x=p, xs=64, r=None, rs=0, ty=1, w=p, eps=1e-6, rows=3, D=64, out=q, sc=q):
        return f(x, xs, r, rs, ty, w, eps, rows, D, out, sc, None)
    for bad in (dict(ty=2), dict(rows=-1), dict(D=0), dict(xs=63), dict(r=q, rs=63), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(out=None), dict(sc=None),
                dict(r=p, rs=64), dict(x=ctypes.c_void_p(257)), dict(sc=ctypes.c_void_p(258)), dict(out=p),
                dict(r=q, rs=64)):
        assert norm(**bad) == INVALID, bad
    assert norm(D=65537, xs=65537) == UNSUPPORTED
    assert norm(rows=0) == OK


def test_matmul_refusals():
    f = _lib.load().gdn_fp8_matmul

    def mm(a=p, lda=64, sa=p, w=p, ldw=64, sw=p, M=3, N=5, K=64, out=q, ty=1):
        return f(a, lda, sa, w, ldw, sw, M, N, K, out, ty, None)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(lda=63), dict(ldw=63), dict(a=None), dict(w=None),
                dict(sa=None), dict(sw=None), dict(out=None), dict(ty=3), dict(sa=ctypes.c_void_p(258)),
                dict(out=ctypes.c_void_p(513)), dict(out=p), dict(a=q)):
        assert mm(**bad) == INVALID, bad
    assert mm(M=0) == OK
    assert mm(M=1 << 40) == UNSUPPORTED
    assert mm(N=(1 << 30) + 1) == UNSUPPORTED
    assert mm(K=(1 << 30) + 1, lda=1 << 31, ldw=1 << 31) == UNSUPPORTED


def test_the_binding_refuses_host_tensors():
    t = torch.zeros(2, 128)
    with pytest.raises(ValueError):
        gdn.rmsnorm_fp8(t, torch.ones(128))
    with pytest.raises(ValueError):
        gdn.fp8_matmul(t.to(torch.float8_e4m3fn), t, t.to(torch.float8_e4m3fn), t)
    x = torch.zeros(1, 4, 2, 32)
    with pytest.raises(ValueError):
        gdn.ssm_scan(x, x[..., 0], x, x, t[0, :2], t[0, :2])
    with pytest.raises(ValueError):
        gdn.ssm_decode_step(torch.zeros(2, 192).bfloat16(), t, t, t, t, t, t, 2, 2, 32, 32)


def test_definitions_against_closed_forms():
    rng = np.random.default_rng(3)
    x, B, C = rng.normal(size=(1, 6, 2, 32)), rng.normal(size=(1, 6, 1, 32)), rng.normal(size=(1, 6, 1, 32))
    dt, none = rng.normal(size=(1, 6, 2)), np.full(2, -np.inf)
    # no decay (A = 0): y_t = sum_s dt_s (C_t . B_s) x_s
    y, hT, _ = layer.ssm_scan(x, dt, B, C, none, np.zeros(2))
    d = np.log1p(np.exp(dt[0]))
    ref = np.einsum("ts,sh,shp->thp", np.tril(C[0, :, 0] @ B[0, :, 0].T), d, x[0])
    assert np.allclose(y[0], ref, rtol=1e-12, atol=1e-12)
    assert np.allclose(hT[0], np.einsum("sn,sh,shp->hnp", B[0, :, 0], d, x[0]))
    # the step is one more token of the scan (W = 1, unit taps, no activation)
    A, b, D = rng.normal(size=2), rng.normal(size=2), rng.normal(size=2)
    y, hT, _ = layer.ssm_scan(x, dt, B, C, A, b, D=D)
    _, h5, _ = layer.ssm_scan(x[:, :5], dt[:, :5], B[:, :5], C[:, :5], A, b, D=D)
    row = np.concatenate([x[0, 5].ravel(), B[0, 5].ravel(), C[0, 5].ravel()])[None]
    ys, st, *_ = layer.ssm_decode_step(row, dt[0, 5:], np.ones((128, 1)), np.zeros((1, 128, 0)), A, b, h5, 2, 1,
                                      32, 32, D=D, activation=False)
    assert np.allclose(ys[0], y[0, 5]) and np.allclose(st[0], hT[0])


def test_scan_workspace_is_that_of_the_device(monkeypatch):
    # the size depends on the device's SMs: it is asked for with the call's device current, and one
    # device's answer is not given for another
    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Lib:
        @staticmethod
        def gdn_ssm_scan_workspace_size(*sizes):
            return 1000 + now[0]

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(_lib, "load", Lib)
    sizes = (3, 12345, 6, 3, 64, 64)
    assert gdn.ssm_scan_workspace_size(*sizes) == 1000
    now[0] = 1
    assert gdn.ssm_scan_workspace_size(*sizes) == 1001
    assert gdn.ssm_scan_workspace_size(*sizes, device="cuda:0") == 1000 and now[0] == 1
    assert gdn.ssm_scan_workspace_size(*sizes, device=torch.device("cuda", 2)) == 1002
    gdn.api._scan_workspace.cache_clear()


def test_scan_workspace_of_a_cut_sequence():
    one = dict(B=1, T=4600, H=2, G=1, P=64, N=64, xs=128, dts=2, bs=64, cs=64)
    need = _lib.load().gdn_ssm_scan_workspace_size(1, 4600, 2, 1, 64, 64, 1)
    assert need > 0
    for bad in (dict(ws=None), dict(wsb=0), dict(wsb=need - 1), dict(ws=ctypes.c_void_p(520))):
        assert scan(**one, **bad) == INVALID, bad
    packed = dict(one, cu=p, n_seq=3, h0=p, hT=q)
    need = _lib.load().gdn_ssm_scan_workspace_size(3, 4600, 2, 1, 64, 64, 1)
    assert need > 0
    for bad in (dict(ws=None), dict(wsb=0), dict(ws=ctypes.c_void_p(520))):
        assert scan(**packed, **bad) == INVALID, bad
