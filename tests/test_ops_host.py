"""Refusals of the checkpoint and recurrence entry points (C ABI; no GPU, nothing is enqueued)."""
import os

import pytest

import receptive_field_spatial_amd as R

A, B_, C_, D_, E_, F_ = (0x10000000 * k for k in range(1, 7))   # never dereferenced
INV, UNS, WS = R.WBMM_E_INVALID, R.WBMM_E_UNSUPPORTED, R.WBMM_E_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(R.lib_path()):
        from receptive_field_spatial_amd.build import build
        build(verbose=False)
    return R.load_library()


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), INV), (dict(n=-5), INV), (dict(n=(1 << 35) + 1), UNS), (dict(dtype=2), INV),
    (dict(fmt=2), INV), (dict(fmt=-1), INV), (dict(x=None), INV), (dict(codes=None), INV),
    (dict(scales=None), INV), (dict(x=A + 2), UNS), (dict(x=A + 1, dtype=1), UNS),
    (dict(codes=A + 100), INV), (dict(scales=B_ + 10), INV), (dict(scales=A + 399), INV),
])
def test_ckpt_refusals(lib, kw, want):
    a = dict(x=A, n=100, dtype=0, fmt=0, codes=B_, scales=C_)
    a.update(kw)
    got = lib.wbmm_ckpt_pack(a["x"], a["n"], a["dtype"], a["fmt"], a["codes"], a["scales"], None)
    assert got == want and lib.wbmm_last_error()
    if "scales" in kw and kw["scales"] == B_ + 10:
        return   # two inputs of the inverse may overlap
    got = lib.wbmm_ckpt_unpack(a["codes"], a["scales"], a["n"], a["dtype"], a["fmt"], a["x"], None)
    assert got == want


def bwd(lib, **kw):
    a = dict(B=2, C=3, H=9, W=9, w=4, layout=0, dtype=0, fmt=0, xc=A, xs=A + 0x100000, T=B_, mix=None,
             zc=None, zs=None, dy=C_, dx=D_, dT=E_, dW=None, ws=F_, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_backward_ckpt(a["B"], a["C"], a["H"], a["W"], a["w"], a["layout"], a["dtype"],
                                  a["fmt"], a["xc"], a["xs"], a["T"], a["mix"], a["zc"], a["zs"],
                                  a["dy"], a["dx"], a["dT"], a["dW"], a["ws"], a["wsb"], None)


MIX = dict(mix=B_ + 0x100000, zc=A + 0x200000, zs=A + 0x300000)


@pytest.mark.parametrize("kw,want", [
    (dict(w=0), INV), (dict(w=33), INV), (dict(B=0), INV), (dict(layout=2), INV),
    (dict(dtype=3), INV), (dict(fmt=4), INV), (dict(xc=None), INV), (dict(xs=None), INV),
    (dict(T=None), INV), (dict(dy=None), INV), (dict(mix=MIX["mix"]), INV),
    (dict(zc=MIX["zc"], zs=MIX["zs"]), INV), (dict(MIX, zs=None), INV), (dict(dy=C_ + 2), UNS),
    (dict(dx=D_ + 1, dtype=1), UNS), (dict(dT=E_ + 2), UNS), (dict(dx=C_), INV), (dict(dx=A), INV),
    (dict(dT=B_), INV), (dict(dT=D_ + 4), INV), (dict(MIX, dW=E_ + 8), INV),
    (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=F_ + 16), UNS),
])
def test_backward_ckpt_refusals(lib, kw, want):
    assert bwd(lib, **kw) == want, lib.wbmm_last_error()


def test_backward_ckpt_with_nothing_to_write(lib):
    assert bwd(lib, dx=None, dT=None) == R.WBMM_OK


def test_backward_ckpt_workspace(lib):
    q = lambda **k: lib.wbmm_backward_ckpt_workspace_bytes(*[{**dict(
        B=2, C=3, H=9, W=9, w=4, layout=0, dtype=0, mix=0), **k}[n]
        for n in ("B", "C", "H", "W", "w", "layout", "dtype", "mix")])
    assert q() > 0 and q(mix=1) >= q() and q(dtype=1) > 0
    assert q(w=20) > 2 * 3 * 9 * 9 * 4      # windows above 16 decode x into the workspace
    assert q(B=0) == 0 and q(dtype=7) == 0 and q(w=40) == 0


def fwd(lib, **kw):
    a = dict(outer=4, len=100, inner=6, dtype=0, rev=0, g=A, u=B_, h0=C_, lens=None, nl=0, h=D_,
             hl=E_, st=F_, ws=7 * A, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_scan_forward(a["outer"], a["len"], a["inner"], a["dtype"], a["rev"], a["g"],
                                 a["u"], a["h0"], a["lens"], a["nl"], a["h"], a["hl"], a["st"],
                                 a["ws"], a["wsb"], None)


SCAN = [
    (dict(outer=0), INV), (dict(len=0), INV), (dict(inner=0), INV), (dict(len=-1), INV),
    (dict(dtype=2), INV), (dict(g=None), INV), (dict(u=None), INV), (dict(g=A + 2), UNS),
    (dict(u=B_ + 1, dtype=1), UNS), (dict(lens=8 * A, nl=3), INV), (dict(lens=8 * A, nl=0), INV),
    (dict(lens=8 * A + 2, nl=2), UNS), (dict(len=(1 << 30) + 1), UNS), (dict(outer=1 << 26), UNS),
    (dict(outer=1 << 13, inner=1 << 13), UNS), (dict(outer=1 << 40, inner=1 << 40), UNS),
    (dict(len=1 << 30, inner=1 << 10), UNS),
]
LONG = dict(outer=1, len=100000, inner=8)


@pytest.mark.parametrize("kw,want", SCAN + [
    (dict(h=None), INV), (dict(h=A), INV), (dict(h=B_ + 4), INV), (dict(hl=C_ + 4), INV),
    (dict(hl=D_ + 8), INV), (dict(st=D_ + 4), INV), (dict(h=C_), INV), (dict(st=C_), INV),
    (dict(lens=E_, nl=4), INV), (dict(LONG, ws=None), WS), (dict(LONG, wsb=8), WS),
    (dict(LONG, ws=7 * A + 8), UNS),
])
def test_scan_forward_refusals(lib, kw, want):
    assert fwd(lib, **kw) == want, lib.wbmm_last_error()


def back(lib, **kw):
    a = dict(outer=4, len=100, inner=6, dtype=0, rev=0, fmt=0, g=A, u=B_, us=None, st=C_, h0=None, dh=D_,
             dhl=None, lens=None, nl=0, dg=E_, du=F_, dh0=None, ws=7 * A, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_scan_backward(a["outer"], a["len"], a["inner"], a["dtype"], a["rev"], a["fmt"],
                                  a["g"], a["u"], a["us"], a["st"], a["h0"], a["dh"], a["dhl"], a["lens"],
                                  a["nl"], a["dg"], a["du"], a["dh0"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", SCAN + [
    (dict(h0=8 * A), INV), (dict(st=None, h0=E_), INV), (dict(dh=None), INV),
    (dict(LONG, st=None, wsb=64), WS), (dict(dg=None), INV), (dict(du=None), INV),
    (dict(us=9 * A, fmt=2), INV), (dict(dg=A), INV), (dict(du=E_ + 4), INV), (dict(dg=D_ + 4), INV),
    (dict(du=C_), INV), (dict(us=E_ + 4, fmt=1), INV), (dict(dhl=9 * A, dh0=9 * A), INV),
    (dict(LONG, ws=None), WS), (dict(st=C_ + 2), UNS),
])
def test_scan_backward_refusals(lib, kw, want):
    assert back(lib, **kw) == want, lib.wbmm_last_error()


def test_scan_workspace_rules(lib):
    q = lib.wbmm_scan_forward_workspace_bytes
    assert q(1, 100000, 8) > 0                 # few columns: the axis runs in segments
    assert q(64 * 192, 784, 1) == 0 and q(4, 32768, 1024) >= 0
    assert q(0, 5, 5) == 0 and q(1, 1 << 31, 1) == 0
    for outer, n, inner in [(1, 1, 1), (1, 1 << 30, 1), (3, 12345, 7), (1, 1 << 20, 65)]:
        # the maps stay a small part of the tensor: 12 workgroups per CU at most form them
        assert q(outer, n, inner) <= (8 * 2 * 12 * 256 + 4) * outer * inner


def test_scan_backward_workspace_rules(lib):
    q = lib.wbmm_scan_backward_workspace_bytes
    assert q(64 * 192, 784, 1, 1) == 0
    assert q(64 * 192, 784, 1, 0) == 0                      # one tile holds the axis
    assert q(64, 30000, 192, 0) >= 64 * 192 * 938 * 4       # the states of 30000 steps
    assert q(0, 5, 5, 1) == 0 and q(1, 1 << 31, 1, 0) == 0
