"""Residual RMS norm against the fp64 oracle.

Tolerances. A row's sum of squares is at most 34 roundings deep (24 terms of a lane, 8 joins and a carry;
columns: 32 entries of a wave, 16 waves), half of which reach rstd, 1 / len and the reciprocal root add 3,
y's two products 2: y within 24 half steps of fp32 before its own rounding. dx is made of w dy and h
mean(w dy h), the mean 34 roundings deep, each factor rounded a few times: 48 half steps of the
magnitudes' sum. dw: products of 3 roundings with a factor good to 20, carried sums, one rounding: 32."""
import numpy as np
import pytest

from oracle import block_oracle as K
from receptive_field_spatial_amd import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = K.U
F32, BF16 = torch.float32, torch.bfloat16


def R():
    import receptive_field_spatial_amd as mod
    mod.load_library()
    return mod


def half(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def mk(shape, sigma, seed, dt=F32):
    return torch.from_numpy(synth.normal_f32(shape, sigma, seed)).cuda().to(dt)


def near(got, want, tol):
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


ROWS = [(1, 1), (5, 2), (3, 7), (65, 8), (130, 31), (9, 32), (33, 64), (64, 96), (77, 97), (50, 192), (7, 256),
        (6, 520), (5, 1000), (3, 1536), (4, 1544), (2, 2048), (3, 6144), (2, 6152), (2, 20001)]
COLS = [(1, 1, 2), (2, 3, 5), (3, 8, 32), (1, 96, 3136), (4, 192, 784), (2, 100, 49), (3, 64, 196), (1, 600, 66),
        (2, 257, 96), (2, 513, 64), (1, 2048, 64), (70, 17, 33), (1, 5, 100003)]
SHAPES = [(o, c, 1) for o, c in ROWS] + COLS


def forward_case(o, c, i, dt, res=True, w=True, fmt=None, eps=1e-6, seed=1):
    x, r = mk((o, c, i), 1.0, seed, dt), mk((o, c, i), 2.0, seed + 1, dt) if res else None
    wt = 1 + mk((c,), 0.2, seed + 2) if w else None
    y, s, ck = R().wbmm_rmsnorm_forward(x, 1, residual=r, weight=wt, eps=eps, fmt=fmt)
    t64, y64 = K.norm_forward(f64(x), f64(r) if res else None, f64(wt) if w else None, eps)
    near(f64(y), y64, 24 * U * np.abs(y64) * (1 + half(dt)) + half(dt) * np.abs(y64))
    if res:
        near(f64(s), t64, (half(dt) + 2 * U) * np.abs(t64))
    else:
        assert s is x
    if fmt:
        codes, scales = R().wbmm_ckpt_pack(y, fmt=fmt)
        assert torch.equal(ck[0], codes) and torch.equal(ck[1], scales)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", SHAPES)
def test_forward(o, c, i, dt):
    print(f"\n[case] norm fwd {o}x{c}x{i} {dt}", flush=True)
    forward_case(o, c, i, dt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", [(9, 32, 1), (64, 96, 1), (50, 192, 1), (77, 97, 1), (3, 6144, 1), (2, 6176, 1),
                                   (3, 8, 32), (1, 96, 3136), (4, 192, 784), (2, 257, 96), (2, 513, 64), (5, 3, 34)])
def test_forward_with_codes(o, c, i, dt, fmt):
    print(f"\n[case] norm codes {o}x{c}x{i} {dt} {fmt}", flush=True)
    forward_case(o, c, i, dt, fmt=fmt, seed=4)


@pytest.mark.parametrize("res,w", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("o,c,i", [(50, 192, 1), (77, 97, 1), (2, 100, 49), (2, 6152, 1), (1, 600, 66)])
def test_forward_without(o, c, i, res, w):
    forward_case(o, c, i, F32, res=res, w=w)
    forward_case(o, c, i, BF16, res=res, w=w, eps=1e-3)


def backward_case(o, c, i, dt, ds=True, w=True, seed=9, eps=1e-6):
    s, dy = mk((o, c, i), 2.0, seed, dt), mk((o, c, i), 1.0, seed + 1, dt)
    g = mk((o, c, i), 1.0, seed + 2, dt) if ds else None
    wt = 1 + mk((c,), 0.2, seed + 3) if w else None
    dx, dw = R().wbmm_rmsnorm_backward(s, dy, 1, weight=wt, ds=g, eps=eps)
    wdx, wdw, mag, wmag = K.norm_backward(f64(s), f64(dy), f64(g) if ds else None, f64(wt) if w else None, eps)
    near(f64(dx), wdx, 48 * U * mag * (1 + half(dt)) + half(dt) * np.abs(wdx))
    if w:
        near(f64(dw), wdw, 32 * U * wmag + U * np.abs(wdw))
    else:
        assert dw is None
    return s, dy, g, wt, dx, dw


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", SHAPES)
def test_backward(o, c, i, dt):
    print(f"\n[case] norm bwd {o}x{c}x{i} {dt}", flush=True)
    backward_case(o, c, i, dt)


@pytest.mark.parametrize("ds,w", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("o,c,i", [(3000, 192, 1), (77, 97, 1), (40, 100, 49), (2, 6152, 1), (1, 600, 66)])
def test_backward_without(o, c, i, ds, w):
    backward_case(o, c, i, F32, ds=ds, w=w)
    backward_case(o, c, i, BF16, ds=ds, w=w, eps=1e-3)


@pytest.mark.parametrize("o,c,i", [(3000, 96, 1), (600, 33, 1), (700, 6152, 1), (1100, 12, 65), (3, 40, 40000)])
def test_backward_over_many_rows(o, c, i):
    """More sets of rows than workgroups; partial outputs equal the whole call's; the same twice."""
    print(f"\n[case] norm bwd many {o}x{c}x{i}", flush=True)
    s, dy, g, wt, dx, dw = backward_case(o, c, i, F32)
    a, none = R().wbmm_rmsnorm_backward(s, dy, 1, weight=wt, ds=g, dweight=False)
    none2, b = R().wbmm_rmsnorm_backward(s, dy, 1, weight=wt, ds=g, dx=False)
    again = R().wbmm_rmsnorm_backward(s, dy, 1, weight=wt, ds=g)
    assert none is None and none2 is None
    assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("o,c,i", [(200000, 8, 1), (2, 8, 200000)])
def test_weight_gradient_of_equal_terms(o, c, i):
    """Terms of one sign, 200000 to a sum."""
    s, dy = torch.ones(o, c, i, device="cuda"), torch.full((o, c, i), 0.1, device="cuda")
    _, dw = R().wbmm_rmsnorm_backward(s, dy, 1, weight=torch.ones(c, device="cuda"), eps=0.0)
    n = o * i
    want = np.float64(np.float32(0.1)) * n
    assert np.all(np.abs(f64(dw) - want) <= 32 * U * want)


@pytest.mark.parametrize("o,c,i", [(50, 192, 1), (4, 192, 784), (3, 2048, 1), (2, 100, 49)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_any_alignment(o, c, i, dt):
    """Every buffer one element off: the same results as aligned ones give."""
    n, M = o * c * i, R()

    def off(t):
        flat = torch.empty(t.numel() + 9, dtype=t.dtype, device="cuda")
        v = flat[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    x, r, w = mk((o, c, i), 1.0, 1, dt), mk((o, c, i), 2.0, 2, dt), 1 + mk((c,), 0.2, 3)
    y, s, ck = M.wbmm_rmsnorm_forward(x, 1, residual=r, weight=w, fmt="int8")
    yo, so = off(y), off(s)
    co, sc = off(ck[0]), off(ck[1])
    y2, s2, ck2 = M.wbmm_rmsnorm_forward(off(x), 1, residual=off(r), weight=off(w), fmt="int8", y=yo.zero_(),
                                         s=so.zero_(), codes=co.zero_(), scales=sc.zero_())
    tol = 48 * U * y.float().abs() + half(dt) * 2 * y.float().abs()
    assert torch.all((y2.float() - y.float()).abs() <= tol) and torch.equal(s2, s)
    codes, scales = M.wbmm_ckpt_pack(y2, fmt="int8")
    assert torch.equal(ck2[0], codes) and torch.equal(ck2[1], scales)
    dy, g = mk((o, c, i), 1.0, 5, dt), mk((o, c, i), 1.0, 6, dt)
    dx, dw = M.wbmm_rmsnorm_backward(s, dy, 1, weight=w, ds=g)
    dx2, dw2 = M.wbmm_rmsnorm_backward(off(s), off(dy), 1, weight=off(w), ds=off(g), dx=off(dx).zero_(),
                                       dweight=off(dw).zero_())
    wdx, wdw, mag, wmag = K.norm_backward(f64(s), f64(dy), f64(g), f64(w), 1e-6)
    near(f64(dx2), wdx, 48 * U * mag * 1.01 + half(dt) * np.abs(wdx))
    near(f64(dw2), wdw, 33 * U * wmag)


@pytest.mark.parametrize("shape,dim", [((2, 6, 5, 7), 1), ((2, 5, 7, 6), 3), ((2, 5, 7, 6), -1), ((4, 6), 1)])
def test_maps_in_both_layouts(shape, dim):
    x, r = mk(shape, 1.0, 1), mk(shape, 1.0, 2)
    w = 1 + mk((6,), 0.2, 3)
    y, s, _ = R().wbmm_rmsnorm_forward(x, dim, residual=r, weight=w)
    t = (x + r).double()
    want = t / torch.sqrt(t.square().mean(dim, keepdim=True) + 1e-6)
    want = want * w.double().view([-1 if d == dim % len(shape) else 1 for d in range(len(shape))])
    assert torch.all((y.double() - want).abs() <= 25 * U * want.abs())


@pytest.mark.parametrize("o,c,i", [(50, 192, 1), (2, 6152, 1), (4, 96, 64), (1, 600, 66)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_sum_in_place(o, c, i, dt):
    x, r, w = mk((o, c, i), 1.0, 1, dt), mk((o, c, i), 2.0, 2, dt), 1 + mk((c,), 0.2, 3)
    y, s, _ = R().wbmm_rmsnorm_forward(x, 1, residual=r, weight=w)
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        y2, s2, _ = R().wbmm_rmsnorm_forward(a, 1, residual=b, weight=w, s=a if target == "x" else b)
        assert torch.equal(y2, y) and torch.equal(s2, s)
        assert torch.equal(b, r) if target == "x" else torch.equal(a, x)


@pytest.mark.parametrize("o,c,i", [(130, 192, 1), (2, 96, 130), (5, 6200, 1), (1, 600, 66)])
def test_infinities_and_nan_stay_in_their_row(o, c, i):
    x, dy = mk((o, c, i), 1.0, 1), mk((o, c, i), 1.0, 2)
    w = 1 + mk((c,), 0.2, 3)
    y0, dx0 = R().wbmm_rmsnorm_forward(x, 1, weight=w)[0], R().wbmm_rmsnorm_backward(x, dy, 1, weight=w)[0]
    x[0, 3, 0], x[o - 1, 5, i - 1] = float("nan"), float("inf")
    y, dx = R().wbmm_rmsnorm_forward(x, 1, weight=w)[0], R().wbmm_rmsnorm_backward(x, dy, 1, weight=w)[0]
    hit = torch.zeros(o, i, dtype=torch.bool, device="cuda")
    hit[0, 0] = hit[o - 1, i - 1] = True
    m = hit[:, None, :].expand(o, c, i)
    assert torch.equal(y[~m], y0[~m]) and torch.equal(dx[~m], dx0[~m])
    assert y[0, :, 0].isnan().all() and y[o - 1, 5, i - 1].isnan()


def test_weight_gradient_without_a_weight():
    """A tensor given is written: the gradient of a weight of ones."""
    s, dy = mk((50, 64, 1), 2.0, 1), mk((50, 64, 1), 1.0, 2)
    dw = torch.zeros(64, device="cuda")
    dx, got = R().wbmm_rmsnorm_backward(s, dy, 1, dweight=dw)
    want = R().wbmm_rmsnorm_backward(s, dy, 1, weight=torch.ones(64, device="cuda"))
    assert got is dw and torch.equal(dw, want[1]) and torch.equal(dx, want[0])
    assert R().wbmm_rmsnorm_backward(s, dy, 1)[1] is None


def test_refused_tensors():
    M = R()
    x, w = mk((4, 6, 8), 1.0, 1), torch.ones(6, device="cuda")
    for kw in (dict(residual=x.bfloat16()), dict(residual=x[:2]), dict(weight=w[:5]), dict(weight=w.double()),
               dict(y=x), dict(residual=x.cpu()), dict(codes=x), dict(fmt="int4"), dict(s=x.transpose(0, 1))):
        with pytest.raises(M.WbmmError):
            M.wbmm_rmsnorm_forward(x, 1, **{"weight": w, **kw})
    for bad in (x.half(), x.cpu(), x.transpose(0, 2)):
        with pytest.raises(M.WbmmError):
            M.wbmm_rmsnorm_forward(bad, 1)
    with pytest.raises(M.WbmmError):
        M.wbmm_rmsnorm_forward(x, 3)
    for kw in (dict(dx=x), dict(ds=x[0]), dict(weight=torch.ones(7, device="cuda")),
               dict(weight=w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(M.WbmmError):
            M.wbmm_rmsnorm_backward(x, x.clone(), 1, **kw)


def test_zero_rows():
    x = torch.zeros(4, 64, 1, device="cuda")
    y, _, _ = R().wbmm_rmsnorm_forward(x, 1, eps=1e-6)
    assert torch.equal(y, x)
    dx, dw = R().wbmm_rmsnorm_backward(x, torch.ones_like(x), 1, weight=torch.ones(64, device="cuda"), eps=1e-4)
    assert torch.allclose(dx, torch.full_like(dx, 100.0), rtol=1e-6) and torch.all(dw == 0)


@pytest.mark.parametrize("o,c,i", [(33, 64, 1), (77, 97, 1), (3, 17, 100), (2, 600, 66), (2, 6152, 1)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_nothing_else_is_written(o, c, i, dt):
    n, pad, M = o * c * i, 64, R()
    x, r, w = mk((o, c, i), 1.0, 1, dt), mk((o, c, i), 2.0, 2, dt), 1 + mk((c,), 0.2, 3)

    def guarded(count, t):
        flat = torch.full((count + 2 * pad,), 77 if t == torch.uint8 else 3.0, dtype=t, device="cuda")
        return flat, flat[pad:pad + count]

    bufs = [guarded(n, dt), guarded(n, dt), guarded(n, torch.uint8), guarded(-(-n // 32), torch.uint8),
            guarded(n, dt), guarded(c, F32)]
    ws = guarded(M.wbmm_rmsnorm_backward_workspace_bytes(o, c, i), torch.uint8)
    M.wbmm_rmsnorm_forward(x, 1, residual=r, weight=w, y=bufs[0][1].view(o, c, i), s=bufs[1][1].view(o, c, i),
                           fmt="e4m3", codes=bufs[2][1].view(o, c, i), scales=bufs[3][1])
    M.wbmm_rmsnorm_backward(x, r, 1, weight=w, dx=bufs[4][1].view(o, c, i), dweight=bufs[5][1], workspace=ws[1])
    for flat, _ in bufs + [ws]:
        fill = 77 if flat.dtype == torch.uint8 else 3.0
        assert torch.all(flat[:pad] == fill) and torch.all(flat[-pad:] == fill)


def test_offsets_past_32_bits():
    """Maps of 4.3e9 bytes: their last rows and columns."""
    c, n = 1024, (1 << 21) + 1500
    x = torch.empty(n, c, dtype=BF16, device="cuda").normal_()
    w = 1 + mk((c,), 0.2, 3)
    y, _, _ = R().wbmm_rmsnorm_forward(x, 1, weight=w)
    dx, _ = R().wbmm_rmsnorm_backward(x, y, 1, weight=w, dweight=False)

    def check(cut):
        want = K.norm_forward(cut(x), None, f64(w), 1e-6)[1]
        near(cut(y), want, (24 * U + 1.01 * half(BF16)) * np.abs(want))
        wdx, _, mag, _ = K.norm_backward(cut(x), cut(y), None, f64(w), 1e-6)
        near(cut(dx), wdx, 49 * U * mag + half(BF16) * np.abs(wdx))

    check(lambda t: f64(t[-1600:])[..., None])
    del x, y, dx
    x = torch.empty(3, 1100, 700000, dtype=BF16, device="cuda").normal_()
    w = 1 + mk((1100,), 0.2, 4)
    y, _, _ = R().wbmm_rmsnorm_forward(x, 1, weight=w)
    dx, _ = R().wbmm_rmsnorm_backward(x, y, 1, weight=w, dweight=False)
    check(lambda t: f64(t[2:, :, -1000:]))


def test_replayed_and_on_another_stream():
    M = R()
    x, r, dy = mk((4, 192, 784), 1.0, 1, BF16), mk((4, 192, 784), 1.0, 2, BF16), mk((4, 192, 784), 1.0, 3, BF16)
    w = 1 + mk((192,), 0.2, 4)

    def step():
        y, s, ck = M.wbmm_rmsnorm_forward(x, 1, residual=r, weight=w, fmt="e4m3")
        return (y, s, *ck, *M.wbmm_rmsnorm_backward(s, dy, 1, weight=w, ds=y))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(mk((4, 192, 784), 1.0, 20 + k, BF16))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = M.wbmm_rmsnorm_forward(x, 1, residual=r, weight=w, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, want[0])


EXACT = [(50, 192, 1), (9, 32, 1), (77, 97, 1), (3, 1544, 1), (2, 6152, 1), (4, 192, 66), (2, 8, 33), (2, 100, 49),
         (1, 600, 66), (2, 257, 96)]


def to_the_last_bit(got, want, dt):
    """y is formed in fp64 and rounded to fp32, and from there to bf16: off by half a step of its own type, and in
    bf16 by as much more as a value next to a tie moves in fp32, 2^-17 of the half step; twice the fp64 part
    (34 roundings of 2^-53) on top. NaN where the oracle has it, infinite past the type's range."""
    bits = 24 if dt == F32 else 8
    with np.errstate(all="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(want))), -126)
        e[want == 0] = -126
    half_step = 2.0 ** (e - bits)
    past = np.abs(want) >= (2 - 2.0 ** -bits) * 2.0 ** 127
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[past], np.copysign(np.inf, want[past]))
    rest = ~past & ~nan
    more = 2.0 ** -20 if dt == F32 else 2.0 ** -15
    bad = np.abs(got[rest] - want[rest]) > half_step[rest] * (1 + more)
    assert not bad.any(), (got[rest][bad][:5], want[rest][bad][:5])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", EXACT)
def test_forward_to_the_last_bit(o, c, i, dt):
    x, wt = mk((o, c, i), 1.0, 31, dt), 1 + mk((c,), 0.2, 32)
    y = R().wbmm_rmsnorm_forward(x, 1, weight=wt)[0]
    to_the_last_bit(f64(y), K.norm_forward(f64(x), None, f64(wt), float(np.float32(1e-6)))[1], dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", EXACT)
def test_forward_with_extreme_weights_and_rows(o, c, i, dt):
    """Infinite and NaN weights, products of rstd and weight beyond fp32 in either direction, rows whose rstd is, rows of
    zeros: what the formula gives, in its own element."""
    print(f"\n[case] norm extremes {o}x{c}x{i} {dt}", flush=True)
    x, wt = mk((o, c, i), 1.0, 33, dt), 1 + mk((c,), 0.2, 34)
    few = [float("inf"), 3e38, -float("inf"), 1e-30, 0.0, float("nan"), -3e38, 2e-38]
    wt[:8] = torch.tensor(few)
    rows = x.permute(0, 2, 1).reshape(-1, c)
    n = rows.shape[0]
    for k, f in enumerate((1e-20, 1e20, 3e-39, 0.0, 1e30)):
        rows[k * n // 7 + n // 9] *= f
    x = rows.view(o, i, c).permute(0, 2, 1).contiguous()
    for eps in (0.0, 1e-6):
        y = R().wbmm_rmsnorm_forward(x, 1, weight=wt, eps=eps)[0]
        with np.errstate(all="ignore"):
            want = K.norm_forward(f64(x), None, f64(wt), float(np.float32(eps)))[1]     # the call takes a float
        to_the_last_bit(f64(y), want, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("o,c,i", EXACT + [(2, 20001, 1), (3, 17, 100), (1, 2048, 64)])
def test_backward_of_extreme_rows(o, c, i, dt):
    """Rows of 1e18 to 1e38 and of 1e-20 to the subnormal numbers, whose squares are past fp32's range: as good as any
    other row (their sums are fp64). The bounds are those of the other rows; what is subnormal in the result
    may be off by one of its steps."""
    print(f"\n[case] norm bwd extremes {o}x{c}x{i} {dt}", flush=True)
    s, dy = mk((o, c, i), 1.0, 35, dt), mk((o, c, i), 1.0, 36, dt)
    wt = 1 + mk((c,), 0.2, 37)
    rows, g = (t.permute(0, 2, 1).reshape(-1, c) for t in (s, dy))
    n = rows.shape[0]
    for r, f in {k * n // 7 + n // 9: f for k, f in enumerate((1e18, 2e19, 1e38 / 6, 1e-20, 1e-30, 3e-39))}.items():
        rows[r] *= f
        g[r] *= 1e-6 if f < 1 else 1.0
    s, dy = (t.view(o, i, c).permute(0, 2, 1).contiguous() for t in (rows, g))
    for eps in (0.0, 1e-6):
        dx, dw = R().wbmm_rmsnorm_backward(s, dy, 1, weight=wt, eps=eps)
        wdx, wdw, mag, wmag = K.norm_backward(f64(s), f64(dy), None, f64(wt), float(np.float32(eps)))
        near(f64(dx), wdx, 48 * U * mag * (1 + half(dt)) + half(dt) * np.abs(wdx) + 2.0 ** (-149 if dt == F32 else -133))
        near(f64(dw), wdw, 32 * U * wmag + U * np.abs(wdw))


@pytest.mark.parametrize("o,c,i", [(20000, 96, 1), (20000, 33, 1), (700, 6152, 1), (70, 12, 650), (3, 40, 40000), (40, 600, 66)])
def test_infinite_gradients_in_the_weights_sums(o, c, i):
    """dweight of an entry is the sum of its terms: infinite where one is, NaN where two cancel, the same as before
    everywhere else."""
    s, dy, w = mk((o, c, i), 1.0, 41), mk((o, c, i), 1.0, 42), torch.ones(c, device="cuda")
    inf = float("inf")
    for e, at in ((3, (0, 0)), (5, (o - 1, i - 1)), (7, (1, 0)), (7, (o - 2, i - 1))):
        s[at[0], e, at[1]] = 1.0
    clean = R().wbmm_rmsnorm_backward(s, dy, 1, weight=w, dx=False)[1]
    dy[0, 3, 0], dy[o - 1, 5, i - 1] = inf, -inf
    dy[1, 7, 0], dy[o - 2, 7, i - 1] = inf, -inf
    got = R().wbmm_rmsnorm_backward(s, dy, 1, weight=w, dx=False)[1]
    assert got[3] == inf and got[5] == -inf and got[7].isnan()
    rest = [e for e in range(c) if e not in (3, 5, 7)]
    assert torch.equal(got[rest], clean[rest])
