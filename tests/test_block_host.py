"""Refusals of the norm, AdamW and delta rule entry points (C ABI; no GPU, nothing is enqueued)."""
import ctypes
import os

import pytest

import receptive_field_spatial_amd as R

A, B_, C_, D_, E_, F_ = (0x10000000 * k for k in range(1, 7))   # never dereferenced
G_, H_, I_, J_, K_, L_, M_ = (0x10000000 * k for k in range(7, 14))
INV, UNS, WS = R.WBMM_E_INVALID, R.WBMM_E_UNSUPPORTED, R.WBMM_E_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(R.lib_path()):
        from receptive_field_spatial_amd.build import build
        build(verbose=False)
    return R.load_library()


SIZES = [(dict(o=0), INV), (dict(n=0), INV), (dict(i=-1), INV), (dict(n=(1 << 20) + 1), UNS),
         (dict(o=(1 << 25) + 1, n=2), UNS), (dict(o=1 << 13, i=1 << 13, n=2), UNS), (dict(o=1 << 40, i=1 << 40), UNS),
         (dict(o=(1 << 23) + 1, n=1537), UNS), (dict(o=1 << 25, n=1 << 12, i=1), UNS), (dict(dt=2), INV),
         (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV)]


def norm_fwd(lib, **kw):
    a = dict(o=4, n=96, i=50, dt=0, eps=1e-6, x=A, r=B_, w=C_, s=D_, y=E_, fmt=0, c=None, sc=None)
    a.update(kw)
    return lib.wbmm_rmsnorm_forward(a["o"], a["n"], a["i"], a["dt"], a["eps"], a["x"], a["r"], a["w"], a["s"],
                                    a["y"], a["fmt"], a["c"], a["sc"], None)


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(x=None), INV), (dict(y=None), INV), (dict(c=F_), INV), (dict(sc=F_), INV), (dict(c=F_, sc=G_, fmt=2), INV),
    (dict(x=A + 2), UNS), (dict(r=B_ + 1, dt=1), UNS), (dict(w=C_ + 2), UNS), (dict(s=D_ + 2), UNS),
    (dict(y=E_ + 1, dt=1), UNS), (dict(y=A), INV), (dict(y=B_ + 4), INV), (dict(s=A + 4), INV), (dict(s=E_ + 4), INV),
    (dict(y=C_), INV), (dict(c=E_, sc=G_), INV), (dict(c=F_, sc=F_ + 5), INV), (dict(c=A, sc=G_), INV),
])
def test_norm_forward_refusals(lib, kw, want):
    assert norm_fwd(lib, **kw) == want and lib.wbmm_last_error()


def norm_bwd(lib, **kw):
    a = dict(o=4, n=96, i=50, dt=0, eps=1e-6, s=A, w=B_, dy=C_, ds=D_, dx=E_, dw=F_, ws=G_, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_rmsnorm_backward(a["o"], a["n"], a["i"], a["dt"], a["eps"], a["s"], a["w"], a["dy"], a["ds"],
                                     a["dx"], a["dw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(s=None), INV), (dict(dy=None), INV), (dict(s=A + 2), UNS), (dict(ds=D_ + 1, dt=1), UNS), (dict(dx=E_ + 2), UNS),
    (dict(dw=F_ + 2), UNS), (dict(w=B_ + 1), UNS), (dict(dx=A), INV), (dict(dx=C_ + 4), INV), (dict(dx=D_), INV),
    (dict(dw=B_), INV), (dict(dw=E_ + 8), INV), (dict(ws=None), WS), (dict(wsb=64), WS), (dict(ws=G_ + 8), UNS),
])
def test_norm_backward_refusals(lib, kw, want):
    assert norm_bwd(lib, **kw) == want and lib.wbmm_last_error()


def test_norm_nothing_to_write(lib):
    assert norm_bwd(lib, dx=None, dw=None, ws=None) == R.WBMM_OK


def test_norm_workspace(lib):
    q = lib.wbmm_rmsnorm_backward_workspace_bytes
    assert q(4, 96, 50) == 200 * 96 * 8 and q(1 << 20, 96, 1) == 512 * 96 * 8
    assert q(0, 1, 1) == 0 and q(1 << 40, 1, 1) == 0


def tensors(*rows):
    t = (R._AdamwTensor * len(rows))()
    for x, kw in zip(t, rows):
        base = dict(p=A, g=B_, m=C_, v=D_, m_scales=None, v_scales=None, p_bf16=None, n=100, weight_decay=0.0,
                    g_dtype=0)
        base.update(kw)
        for k, v in base.items():
            setattr(x, k, v)
    return t


def plan(lib, rows, count=None, bytes_=None, table=True, chunks=True, off=0):
    t = tensors(*rows)
    buf = ctypes.create_string_buffer(1 << 20)
    at = (ctypes.addressof(buf) + 15) // 16 * 16 + off
    n = ctypes.c_int64(-1)
    got = lib.wbmm_adamw_plan(t, len(rows) if count is None else count, at if table else None,
                              (1 << 20) - 64 if bytes_ is None else bytes_, ctypes.byref(n) if chunks else None)
    return got, n.value


OTHER = dict(p=E_, g=F_, m=G_, v=H_)


@pytest.mark.parametrize("rows,kw,want", [
    ([dict(n=0)], {}, INV), ([dict(n=-4)], {}, INV), ([dict(n=1 << 40)], {}, UNS), ([{}], dict(count=0), INV),
    ([{}], dict(count=1 << 30), UNS),
    ([dict(p=None)], {}, INV), ([dict(g=None)], {}, INV), ([dict(m=None)], {}, INV), ([dict(v=None)], {}, INV),
    ([dict(m_scales=E_)], {}, INV), ([dict(v_scales=E_)], {}, INV), ([dict(g_dtype=2)], {}, INV),
    ([dict(weight_decay=-0.1)], {}, INV), ([dict(weight_decay=float("nan"))], {}, INV), ([dict(p=A + 2)], {}, UNS),
    ([dict(g=B_ + 2)], {}, UNS), ([dict(g=B_ + 1, g_dtype=1)], {}, UNS), ([dict(m=C_ + 1)], {}, UNS),
    ([dict(p_bf16=E_ + 1)], {}, UNS), ([dict(g=A)], {}, INV), ([dict(m=A + 396)], {}, INV), ([dict(v=C_)], {}, INV),
    ([dict(p_bf16=D_ + 100)], {}, INV), ([{}, {}], {}, INV), ([{}, dict(OTHER, m=A + 8)], {}, INV),
    ([{}, dict(OTHER, g=A + 8)], {}, INV), ([{}, dict(OTHER, p=B_)], {}, INV),
    ([dict(m_scales=E_, v_scales=E_ + 3)], {}, INV), ([{}], dict(table=False), INV), ([{}], dict(chunks=False), INV),
    ([{}], dict(bytes_=64), WS), ([{}], dict(off=4), UNS),
])
def test_adamw_plan_refusals(lib, rows, kw, want):
    assert plan(lib, rows, **kw)[0] == want and lib.wbmm_last_error()


def test_adamw_plan_accepts(lib):
    assert plan(lib, [{}, dict(OTHER, g=B_)]) == (0, 2)             # one gradient for two tensors
    assert plan(lib, [dict(n=4096), dict(OTHER, n=4097)]) == (0, 3)
    assert plan(lib, [dict(m=C_ + 1, v=D_ + 3, m_scales=E_, v_scales=E_ + 4)]) == (0, 1)
    assert plan(lib, [dict(p=A + 4)])[0] == 0
    t = tensors({}, OTHER)
    assert lib.wbmm_adamw_plan_bytes(t, 2) == 32 + 2 * 80 + 2 * 4
    assert lib.wbmm_adamw_plan_bytes(t, 0) == 0 and lib.wbmm_adamw_plan_bytes(None, 1) == 0
    assert ctypes.sizeof(R._AdamwTensor) == 80


def step(lib, **kw):
    a = dict(t=A, n=3, c=5, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, sd=None, lf=None, gf=None)
    a.update(kw)
    return lib.wbmm_adamw_step(a["t"], a["n"], a["c"], a["lr"], a["b1"], a["b2"], a["eps"], a["step"], a["sd"],
                               a["lf"], a["gf"], 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=None), INV), (dict(n=0), INV), (dict(c=2), INV), (dict(c=1 << 24), INV), (dict(lr=float("inf")), INV),
    (dict(b1=1.0), INV), (dict(b1=-0.1), INV), (dict(b2=float("nan")), INV), (dict(eps=-1e-8), INV),
    (dict(eps=float("inf")), INV), (dict(step=0), INV), (dict(step=1 << 31), INV), (dict(t=A + 4), UNS),
    (dict(sd=B_ + 2), UNS), (dict(lf=B_ + 1), UNS), (dict(gf=B_ + 2), UNS),
])
def test_adamw_step_refusals(lib, kw, want):
    assert step(lib, **kw) == want and lib.wbmm_last_error()


def delta_fwd(lib, **kw):
    a = dict(B=2, L=100, Hk=2, H=4, dk=32, dv=24, dt=0, rev=0, scale=0.2, q=A, k=B_, v=C_, g=D_, be=E_, s0=F_,
             lens=None, o=G_, sl=H_, st=I_, ws=J_, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_delta_forward(a["B"], a["L"], a["Hk"], a["H"], a["dk"], a["dv"], a["dt"], a["rev"], a["scale"],
                                  a["q"], a["k"], a["v"], a["g"], a["be"], a["s0"], a["lens"], a["o"], a["sl"],
                                  a["st"], a["ws"], a["wsb"], None)


DELTA = [(dict(B=0), INV), (dict(L=0), INV), (dict(Hk=0), INV), (dict(H=3), INV), (dict(dk=0), INV), (dict(dv=-1), INV),
         (dict(dk=129), UNS), (dict(dv=129), UNS), (dict(L=(1 << 28) + 1), UNS), (dict(B=1 << 22), UNS),
         (dict(B=1 << 50, H=1 << 20), UNS), (dict(H=1 << 18, Hk=1 << 18), UNS), (dict(dt=2), INV),
         (dict(scale=float("nan")), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV),
         (dict(g=None), INV), (dict(be=None), INV), (dict(q=A + 2), UNS), (dict(v=C_ + 1, dt=1), UNS),
         (dict(g=D_ + 2), UNS), (dict(s0=F_ + 2), UNS), (dict(lens=K_ + 2), UNS), (dict(ws=None), WS), (dict(wsb=64), WS),
         (dict(ws=J_ + 8), UNS)]


@pytest.mark.parametrize("kw,want", DELTA + [
    (dict(o=None), INV), (dict(o=C_), INV), (dict(o=A + 4), INV), (dict(sl=F_ + 4), INV), (dict(sl=G_ + 8), INV),
    (dict(st=F_), INV), (dict(st=H_ + 4), INV), (dict(o=G_ + 2), UNS), (dict(st=I_ + 2), UNS), (dict(lens=G_), INV),
])
def test_delta_forward_refusals(lib, kw, want):
    assert delta_fwd(lib, **kw) == want and lib.wbmm_last_error()


def delta_bwd(lib, **kw):
    a = dict(B=2, L=100, Hk=2, H=4, dk=32, dv=24, dt=0, rev=0, scale=0.2, q=A, k=B_, v=C_, g=D_, be=E_, st=I_, s0=None,
             do=F_, dl=None, lens=None, dq=G_, dkey=H_, dval=K_, dg=L_, db=M_, d0=None, ws=J_, wsb=1 << 30)
    a.update(kw)
    return lib.wbmm_delta_backward(a["B"], a["L"], a["Hk"], a["H"], a["dk"], a["dv"], a["dt"], a["rev"], a["scale"],
                                   a["q"], a["k"], a["v"], a["g"], a["be"], a["st"], a["s0"], a["do"], a["dl"],
                                   a["lens"], a["dq"], a["dkey"], a["dval"], a["dg"], a["db"], a["d0"], a["ws"],
                                   a["wsb"], None)


@pytest.mark.parametrize("kw,want", [x for x in DELTA if "s0" not in x[0]] + [
    (dict(do=None), INV), (dict(dq=None), INV), (dict(dkey=None), INV), (dict(dval=None), INV), (dict(dg=None), INV),
    (dict(db=None), INV), (dict(s0=14 * A), INV), (dict(st=None, s0=14 * A + 2), UNS), (dict(st=I_ + 2), UNS),
    (dict(dq=A), INV), (dict(dkey=G_ + 4), INV), (dict(dval=F_), INV), (dict(dg=D_), INV), (dict(db=L_ + 4), INV),
    (dict(d0=I_), INV), (dict(dl=14 * A, d0=14 * A + 4), INV), (dict(dq=G_ + 2), UNS), (dict(d0=15 * A + 2), UNS),
])
def test_delta_backward_refusals(lib, kw, want):
    assert delta_bwd(lib, **kw) == want and lib.wbmm_last_error()


def test_delta_workspaces(lib):
    f, b = lib.wbmm_delta_forward_workspace_bytes, lib.wbmm_delta_backward_workspace_bytes
    assert f(2, 8, 1, 2, 64, 64, 0) == 0 and f(2, 9, 1, 2, 64, 64, 0) > 0      # single steps need none
    assert f(2, 9, 1, 2, 64, 64, 1) < f(2, 9, 1, 2, 64, 64, 0)
    assert f(1, 640, 1, 1, 64, 64, 1) == 10 * f(1, 64, 1, 1, 64, 64, 1)
    with_, without = b(1, 640, 1, 1, 64, 64, 0, 1), b(1, 640, 1, 1, 64, 64, 0, 0)
    assert without - with_ == 10 * 64 * 64 * 4
    assert f(0, 9, 1, 2, 64, 64, 0) == 0 and b(2, 9, 1, 2, 200, 64, 0, 1) == 0 and f(2, 9, 1, 2, 64, 64, 5) == 0
