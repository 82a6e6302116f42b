"""The gated linear recurrence on the GPU against the fp64 oracle, element by element, within the
bound that the oracle carries along for fp32 arithmetic, plus half a step of the output's type."""
import numpy as np
import pytest

from oracle import ops_oracle as Q
from receptive_field_spatial_amd import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def R():
    import receptive_field_spatial_amd as mod
    mod.load_library()
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def draw(shape, bf16, seed, spread=3.0):
    O, L, I = shape
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(shape) + rng.uniform(-1, 2 * spread, (O, 1, I))
    u, dh = rng.standard_normal(shape), rng.standard_normal(shape)
    h0, dl = rng.standard_normal((O, I)), rng.standard_normal((O, I))
    arrs = [a.astype(np.float32) for a in (g, u, dh, h0, dl)]
    if bf16:
        arrs[:3] = [synth.round_to_bf16(a) for a in arrs[:3]]
    return arrs


def close(got, want, bound, bf16, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = bound * (1 + half) + half * np.abs(want) + 1e-36
    err = np.abs(got - want)
    worst = np.max(np.where(tol > 0, err / tol, np.where(err > 0, np.inf, 0)))
    print(f"    {what}: worst error/bound {worst:.3f}, max abs {err.max():.2e}", flush=True)
    assert np.all(err <= tol), (what, worst)


def run_case(O, L, I, bf16=False, reverse=False, lens=None, ckpt=None, h0=True, seed=0, arrs=None,
             recompute=False):
    print(f"\n[case] scan {O}x{L}x{I} bf16={bf16} rev={reverse} lens={lens} ckpt={ckpt}", flush=True)
    shape = (O, L, I)
    g, u, dh, s0, dl = arrs or draw(shape, bf16, seed)
    dt = torch.bfloat16 if bf16 else torch.float32
    gd, ud, dd = (dev(a).to(dt) for a in (g, u, dh))
    n = None
    ln = None
    if lens is not None:
        ln = dev(np.asarray(lens, np.int32))
        n = np.clip(np.repeat(lens, O // len(lens)), 0, L)
        # positions past the end may hold anything
        for o in range(O):
            for t in (gd, ud, dd):
                t[o, n[o]:] = float("nan")
        g, u, dh = g.copy(), u.copy(), dh.copy()
        for o in range(O):
            g[o, n[o]:] = u[o, n[o]:] = dh[o, n[o]:] = 0
    st0 = dev(s0) if h0 else None
    h, last, states = R().wbmm_scan_forward(gd, ud, 1, h0=st0, lens=ln, reverse=reverse,
                                            h_last=True, states=True)
    f64 = [a.astype(np.float64) for a in (g, u, dh, s0, dl)]
    wh, wl, wst, bh, bl, bst = Q.scan_forward(f64[0], f64[1], f64[3] if h0 else None, n, reverse,
                                              bf16)
    close(h, wh, bh, bf16, "h")
    close(last, wl, bl, False, "h_last")
    close(states, wst, bst, False, "states")
    kw = dict(u=ud)
    uval = f64[1]
    if ckpt:
        clean = ud.nan_to_num(0.0)
        kw = dict(u_ckpt=R().wbmm_ckpt_pack(clean, fmt=ckpt), fmt=ckpt)
        uval = R().wbmm_ckpt_unpack(*kw["u_ckpt"], fmt=ckpt).double().cpu().numpy()
        if lens is not None:
            for o in range(O):
                uval[o, n[o]:] = 0
        # the oracle is the recurrence on the decoded u: its states, or none (then the call runs
        # it for them)
        states = R().wbmm_scan_forward(gd, dev(uval.astype(np.float32)).to(dt), 1, h0=st0, lens=ln,
                                       reverse=reverse, states=True)[2]
    if recompute:
        states = None
        kw["h0"] = st0
    dg, du, d0 = R().wbmm_scan_backward(gd, states, dd, 1, dh_last=dev(dl), lens=ln,
                                        reverse=reverse, **kw)
    wdg, wdu, wd0, bg, bu, b0 = Q.scan_backward(f64[0], uval, f64[3] if h0 else None, f64[2],
                                                f64[4], n, reverse, bf16)
    close(dg, wdg, bg, bf16, "dg")
    close(du, wdu, bu, bf16, "du")
    close(d0, wd0, b0, False, "dh0")


SHAPES = [
    (1, 1, 1), (3, 1, 5), (7, 1, 1), (1, 2, 1), (2, 5, 1), (5, 8, 1), (9, 9, 1), (4, 16, 1),
    (3, 17, 1), (3, 33, 1), (2, 64, 1), (3, 65, 1), (3, 127, 1), (2, 129, 1), (2, 256, 1),
    (2, 257, 1), (3, 511, 1), (2, 513, 1), (5, 784, 1), (2, 1000, 1), (1, 4097, 1),
    (2, 2, 2), (3, 7, 3), (2, 15, 64), (2, 16, 65), (1, 17, 130), (2, 31, 6), (2, 32, 192),
    (3, 33, 97), (1, 128, 63), (1, 129, 64), (2, 255, 10), (1, 300, 2), (1, 1531, 97),
]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("O,L,I", SHAPES)
def test_scan(O, L, I, bf16, reverse):
    run_case(O, L, I, bf16, reverse, seed=O + L + I)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("O,L,I,lens", [
    (4, 40, 1, [0, 1, 40, 17]), (4, 700, 1, [0, 1, 700, 513]), (4, 90, 7, [0, 1, 90, 33]),
    (4, 300, 66, [300, 0, 16, 129]), (6, 50, 1, [3, 50]), (6, 50, 3, [0, 50, 7]),
    (2, 1, 1, [0, 1]), (2, 1, 4, [1, 0]), (2, 20, 5, [-3, 99]), (3, 5000, 1, [4999, 0, 512]),
    (3, 2600, 10, [2600, 0, 1100]),
])
def test_scan_lengths(O, L, I, lens, bf16, reverse):
    run_case(O, L, I, bf16, reverse, lens=lens, seed=L)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("O,L,I,reverse,lens", [
    (5, 784, 1, False, None), (3, 37, 1, True, None), (3, 37, 1, True, [37, 0, 9]),
    (2, 1001, 1, True, None), (2, 100, 7, False, None), (2, 100, 64, True, [100, 41]),
    (1, 5003, 1, False, None), (1, 2001, 9, True, None),
])
def test_scan_backward_from_checkpoint(O, L, I, reverse, lens, fmt, bf16):
    run_case(O, L, I, bf16, reverse, lens=lens, ckpt=fmt, seed=L)
    run_case(O, L, I, bf16, reverse, lens=lens, ckpt=fmt, seed=L, recompute=True)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("O,L,I,reverse", [
    (300, 50, 7, False), (1000, 40, 40, True), (17, 200, 130, True), (129, 65, 128, False),
    (1, 1000, 1000, False), (2, 700, 2, True), (5000, 300, 1, False), (1, 900, 17, True),
])
def test_scan_many_columns(O, L, I, reverse, bf16):
    """Column groups of every width, with and without columns to spare."""
    run_case(O, L, I, bf16, reverse, seed=3)
    run_case(O, L, I, bf16, reverse, seed=4, lens=[L // 2 + 1], recompute=True)


@pytest.mark.parametrize("shape", [(1, (1 << 23) + 5, 257), (3, (1 << 30) - 3, 1)])
def test_scan_offsets_past_32_bits(shape):
    """More than 4 GiB of bf16: the ends of the long run against runs of the ends alone."""
    O, L, I = shape
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, u, dh = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for t in (g, u, dh):
        t.normal_(generator=gen)
    h, last, st = R().wbmm_scan_forward(g, u, 1, h_last=True, states=True)
    k = (L // 32 - 3) * 32      # a chunk's start near the end
    cut = lambda t, a, b: t[-1:, a:b].contiguous()
    h2, last2, _ = R().wbmm_scan_forward(cut(g, k, L), cut(u, k, L), 1,
                                         h0=st[-1:, k // 32].contiguous(), h_last=True)
    same = lambda a, b: torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)
    assert same(h[-1:, k:], h2) and same(last[-1:], last2)
    dg, du, d0 = R().wbmm_scan_backward(g, st, dh, 1, u=u)
    n = 3000                    # the last sequence's end, and its beginning (the rest forgotten)
    for a, b, keep in ((L - n, L, slice(0, n)), (0, n, slice(0, n - 1000))):
        a = a // 32 * 32
        x, y, z = R().wbmm_scan_backward(cut(g, a, b), None, cut(dh, a, b), 1, u=cut(u, a, b),
                                         h0=st[-1:, a // 32].contiguous())
        assert same(dg[-1:, a:b][:, keep], x[:, keep]) and same(du[-1:, a:b][:, keep], y[:, keep])
    assert torch.allclose(d0[-1:], z, rtol=1e-4, atol=1e-5)
    # the same from a checkpoint of u, whose codes and scales lie as far out
    ck = R().wbmm_ckpt_pack(u)
    u.copy_(R().wbmm_ckpt_unpack(*ck, dtype=torch.bfloat16))
    want = R().wbmm_scan_backward(g, st, dh, 1, u=u, dg=dg, du=du)
    tail = [t[-1:, -4000:].clone() for t in want[:2]]
    dg.zero_(), du.zero_()
    R().wbmm_scan_backward(g, st, dh, 1, u_ckpt=ck, dg=dg, du=du)
    for t, v in zip(tail, (dg, du)):
        assert same(t, v[-1:, -4000:])


def test_scan_more_rows_than_two_waves_each():
    """2^25 rows of two tiles: a workgroup of two waves per row would be a launch of 2^32 threads."""
    O, L = (1 << 25) + 3, 515
    g = torch.empty((O, L, 1), dtype=torch.bfloat16, device="cuda")
    g.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    rows = [0, 1, 77, 1 << 24, (1 << 25) - 1, 1 << 25, O - 2, O - 1]
    f = g[rows].double().cpu().numpy()          # one tensor serves as g, u and dh
    h, last, _ = R().wbmm_scan_forward(g, g, 1, h_last=True)
    wh, wl, _, bh, bl, _ = Q.scan_forward(f, f, bf16=True)
    close(h[rows], wh, bh, True, "h")
    close(last[rows], wl, bl, False, "h_last")
    del h
    dg, du, d0 = R().wbmm_scan_backward(g, None, g, 1, u=g)
    want = Q.scan_backward(f, f, None, f, bf16=True)
    for t, w, b, bf16, name in zip((dg, du, d0), want[:3], want[3:], (True, True, False), ("dg", "du", "dh0")):
        close(t[rows], w, b, bf16, name)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("O,L,I,reverse,lens", [
    (2, 1, 1, False, None), (2, 1, 3, False, [0, 1]), (3, 20, 1, True, None), (2, 600, 1, True, [600, 5]),
    (2, 90, 7, False, None), (2, 33, 64, True, [33, 0]), (1, 9000, 1, True, None), (1, 3001, 4, False, None),
])
def test_scan_backward_without_states(O, L, I, reverse, lens, bf16):
    run_case(O, L, I, bf16, reverse, lens=lens, seed=L, recompute=True)
    run_case(O, L, I, bf16, reverse, lens=lens, seed=L, recompute=True, h0=False)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("O,L,I", [(1, 20000, 1), (2, 9001, 1), (1, 12000, 3), (1, 4097, 192)])
def test_scan_long_few_columns(O, L, I, bf16):
    run_case(O, L, I, bf16, False, seed=1)
    run_case(O, L, I, bf16, True, lens=[L - 700] * O, seed=2, recompute=True)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("O,L,I,lens", [(1, 70001, 1, None), (2, 40000, 1, [40000, 333]),
                                        (1, 70000, 2, [50000]), (1, 33000, 130, None)])
def test_scan_in_segments(O, L, I, lens, bf16):
    """Long axes of few columns run in segments, with the maps' launch before the second."""
    assert R().wbmm_scan_forward_workspace_bytes(O, L, I) > 0
    assert R().wbmm_scan_backward_workspace_bytes(O, L, I, True) > 0
    run_case(O, L, I, bf16, False, lens=lens, seed=1)
    run_case(O, L, I, bf16, True, lens=lens, seed=2, ckpt="int8", recompute=True)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("O,L,I,reverse,lens", [
    (3, 40, 32, False, None), (5, 77, 96, True, [77, 0, 1, 16, 50]), (300, 300, 64, True, None),
    (2, 700, 160, False, [700, 333]), (90, 260, 96, False, [260, 100, 17] * 30), (1, 33, 1024, True, None),
    (1, 6000, 192, True, [5000]), (129, 17, 32, False, None),
])
def test_scan_backward_from_checkpoint_whole_groups(O, L, I, reverse, lens, fmt, bf16):
    """Rows of whole groups, so that a group holds one step of 32 columns."""
    run_case(O, L, I, bf16, reverse, lens=lens, seed=L, ckpt=fmt)
    run_case(O, L, I, bf16, reverse, lens=lens, seed=L + 1, ckpt=fmt, recompute=True)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("O,L,I,reverse,lens", [
    (5, 784, 1, False, None), (3, 37, 1, True, [37, 0, 9]), (2, 1001, 1, True, None), (2, 100, 7, False, None),
    (2, 300, 64, True, [300, 41]), (1, 1500, 96, False, None), (1, 9000, 2, False, None), (2, 1, 40, False, None),
])
def test_scan_backward_from_checkpoint_and_the_forwards_states(O, L, I, reverse, lens, fmt, bf16):
    """What a training step keeps: the states of the forward's own u, and u in 8 bits. Every run of 32
    steps starts from its state and goes on with the decoded u."""
    g, u, dh, s0, dl = draw((O, L, I), bf16, L + I)
    dt = torch.bfloat16 if bf16 else torch.float32
    gd, ud, dd = (dev(a).to(dt) for a in (g, u, dh))
    ln = None if lens is None else dev(np.asarray(lens, np.int32))
    n = np.full(O, L) if lens is None else np.repeat(lens, O // len(lens))
    states = R().wbmm_scan_forward(gd, ud, 1, h0=dev(s0), lens=ln, reverse=reverse, states=True)[2]
    ck = R().wbmm_ckpt_pack(ud, fmt=fmt)
    got = R().wbmm_scan_backward(gd, states, dd, 1, u_ckpt=ck, fmt=fmt, dh_last=dev(dl), lens=ln, reverse=reverse)

    def order(a):   # scan order, zeros past the end
        a = a.astype(np.float64).copy()
        for o in range(O):
            a[o, :n[o]] = a[o, :n[o]][::-1 if reverse else 1]
            a[o, n[o]:] = 0
        return a

    f64 = lambda t: t.double().cpu().numpy()
    G_, U_, D_ = order(g), order(f64(R().wbmm_ckpt_unpack(*ck, fmt=fmt))), order(dh)
    _, du, d0, _, bu, b0 = Q.scan_backward(G_, U_, None, D_, dl.astype(np.float64), n, False, bf16)
    c = 1 / (1 + np.exp(G_))
    ea, ec = Q.gate_bounds(G_, bf16)
    grad = du / c                                           # of each step's state
    gerr = bu / c - np.abs(grad) * (ec + 2 * Q.U)
    # the state before every step, and its bound: runs of 32 steps as sequences of their own
    K = Q.CHUNK
    ch = -(-L // K)
    cut = lambda a: np.pad(a, ((0, 0), (0, ch * K - L), (0, 0))).reshape(O * ch, K, I)
    st = f64(states).reshape(O * ch, I)
    nk = np.clip(n[:, None] - K * np.arange(ch), 0, K).reshape(-1)
    h, _, _, hb, _, _ = Q.scan_forward(cut(G_), cut(U_), st, nk, False, bf16)
    join = lambda first, a: np.concatenate([first[:, None], a[:, :-1]], 1).reshape(O, ch * K, I)[:, :L]
    # c (h - u) is formed as c h less the rounded c u: U |u| beside the state's own error, which is none
    # at a run's first step
    prev, perr = join(st, h), join(np.zeros_like(st), hb) + Q.U * np.abs(U_)
    x, w = prev - U_, c / (1 + np.exp(-G_))
    inside = (np.arange(L) < n[:, None])[:, :, None]
    dg = np.where(inside, w * x * grad, 0)
    bg = w * (np.abs(x) * gerr + np.abs(grad) * (perr + np.abs(x) * (ea + ec + 4 * Q.U)))
    back = lambda a: order(np.where(inside, a, 0))          # its own inverse
    close(got[0], back(dg), back(bg), bf16, "dg")
    close(got[1], back(du), back(bu), bf16, "du")
    close(got[2], d0, b0, False, "dh0")


@pytest.mark.parametrize("bf16", [False, True])
def test_scan_in_finer_parts(bf16):
    """Segments whose maps are formed from two parts each, in 15 and 29 column groups."""
    run_case(1, 5000, 900, bf16, False, seed=1)
    run_case(1, 5000, 900, bf16, True, lens=[4100], seed=2, ckpt="e4m3", recompute=True)


@pytest.mark.parametrize("L", [(1 << 24) - 3, (1 << 22) + 5])
def test_scan_one_long_column(L):
    """One column in thousands of maps (2048 of them at 2^24 steps), memories from a step to a million:
    the oracle's sums and bounds, its loop over steps written as a doubling in fp64."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda: torch.randn(L, dtype=torch.float32, device="cuda", generator=gen)
    g = r() + 7 + 7 * torch.sin(torch.arange(L, device="cuda") * (2e-6 * np.pi))
    u, dh = r(), r()

    def scan(a, b):   # h_t = a_t h_{t-1} + b_t
        a, b, d = a.clone(), b.clone(), 1
        while d < L:
            b[d:] = b[d:] + a[d:] * b[:-d]
            a[d:] = a[d:] * a[:-d]
            d *= 2
        return b

    U = Q.U
    x = g.double()
    a, c = torch.sigmoid(x), torch.sigmoid(-x)
    ea = c * (3 * U) + 3 * U
    ec = ea + 4 * U

    def bounds(a, b, eb, ea):   # with S the sum of magnitudes and E the error that has come up
        h, S = scan(a, b), scan(a, b.abs())
        before = torch.cat([S.new_zeros(1), S[:-1]])
        E = scan(a, a * before * (ea + 3 * U) + b.abs() * eb)
        return h, E + 40 * U * S, S

    def near(got, want, bound, what):
        err = (got.double().reshape(want.shape) - want).abs()
        tol = bound * (1 + U) + U * want.abs() + 1e-36
        print(f"    {what}: worst error/bound {(err / tol).max().item():.3f}", flush=True)
        assert torch.all(err <= tol), what

    col = lambda t: t.reshape(1, L, 1)
    h, last, st = R().wbmm_scan_forward(col(g), col(u), 1, h_last=True, states=True)
    wh, bh, _ = bounds(a, c * u.double(), ec + 3 * U, ea)
    near(h, wh, bh, "h")
    near(last, wh[-1:], bh[-1:], "h_last")
    dg, du, d0 = R().wbmm_scan_backward(col(g), st, col(dh), 1, u=col(u))
    # G_t = dh_t + a_{t+1} G_{t+1}
    nxt = torch.cat([a[1:], a.new_zeros(1)]).flip(0)
    eb = torch.cat([ea[1:], ea.new_zeros(1)]).flip(0)
    G, bG, _ = (t.flip(0) for t in bounds(nxt, dh.double().flip(0), 3 * U, eb))
    near(du, c * G, c * (bG + G.abs() * (ec + 2 * U)), "du")
    prev, bp = (torch.cat([t.new_zeros(1), t[:-1]]) for t in (wh, bh))
    xx, w = prev - u.double(), a * c
    near(dg, w * xx * G, w * (xx.abs() * bG + G.abs() * (bp + U * u.double().abs() + xx.abs() * (ea + ec + 4 * U))), "dg")
    near(d0, (a * G)[:1], (a * bG + (a * G).abs() * (ea + 3 * U))[:1], "dh0")


def test_scan_without_initial_state_and_extreme_gates():
    shape = (3, 70, 2)
    arrs = draw(shape, False, 3)
    arrs[0][0, ::3] = 100.0     # a = 1: u ignored
    arrs[0][1, ::5] = -100.0    # a = 0: the state is replaced
    arrs[0][2, 7] = 3e38
    arrs[0][2, 9] = -3e38
    run_case(*shape, h0=False, arrs=arrs)
    flat = [np.ascontiguousarray(a.reshape(1, -1, 1) if a.ndim == 3 else a[:1, :1]) for a in arrs]
    run_case(1, 420, 1, arrs=flat)


def test_scan_gate_infinite():
    g = torch.tensor([0.0, float("inf"), 1.0, float("-inf"), 2.0], device="cuda").reshape(1, 5, 1)
    u = torch.tensor([1.0, 5.0, 1.0, 7.0, 1.0], device="cuda").reshape(1, 5, 1)
    for t in (g, g.expand(1, 5, 2).contiguous()):
        h = R().wbmm_scan_forward(t, u.expand_as(t).contiguous(), 1)[0]
        assert torch.isfinite(h).all()
        assert torch.equal(h[0, 1], h[0, 0])
        # a = 0 to within the least normal number; c = t (1 / (1 + t)) with 1 + t = t: the
        # reciprocal is within one step (2^-23), its product with t and that with u take half a
        # step (2^-24) each
        assert torch.all((h[0, 3] - 7).abs() <= 7 * (2.0 ** -23 + 2 * 2.0 ** -24))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kernel", ["step", "rows", "columns"])
def test_scan_gate_accuracy(kernel, bf16):
    """Sigmoid(g) and sigmoid(-g) as fp32 outputs show them: the state after one step from 1 with u = 0,
    and from 0 with u = 1, is a, and 1 - a.

    Relative error of t = exp(-g): one step of the hardware's exp2, 2 U with U = 2^-24 (the exponent it
    is given is exact, or its rounding is put back), and U for the correction; with the exponent in
    two parts (bf16) the square of the second is left out, z^2 / 2 with z below 7.2e-6 ln(2) |g|,
    2.1e-4 g^2 U. a = 1 / (1 + t) takes (1 - a) of that, U for the sum and U for the reciprocal with
    its Newton step (whose own residue, (2 U)^2, is nothing); c = t a takes a of it, both and U. The
    sums around them multiply by 1 or add 0, and are exact."""
    U = 2.0 ** -24
    if bf16:   # every bf16 value in range, and its negative
        g = np.arange(0x3a80, 0x42ae, dtype=np.uint32) << 16
        g = g.view(np.float32)
    else:
        g = np.exp(np.linspace(np.log(1e-3), np.log(86.9), 20000)).astype(np.float32)
    g = np.concatenate([g, -g, [0]]).astype(np.float32)
    n = g.size
    shape = {"step": (1, 1, n), "rows": (n, 2, 1), "columns": (1, 2, n)}[kernel]
    dt = torch.bfloat16 if bf16 else torch.float32
    gd = dev(g).to(dt)
    if kernel != "step":   # the second step leaves the state alone: a = 1, u = 0
        gd = torch.stack([gd, torch.full_like(gd, 100.0)], 1 if kernel == "rows" else 0)
    gd = gd.reshape(shape).contiguous()
    u = torch.zeros(shape, dtype=dt, device="cuda")
    u[:, 0] = 1
    one = torch.ones(shape[0], shape[2], device="cuda")
    c = R().wbmm_scan_forward(gd, u, 1, h_last=True)[1].double().cpu().numpy().reshape(-1)
    a = R().wbmm_scan_forward(gd, torch.zeros_like(u), 1, h0=one, h_last=True)[1].double().cpu().numpy().reshape(-1)
    x = g.astype(np.float64)
    wa, wc = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    et = 3 + (2.1e-4 * x * x if bf16 else 0)
    ra, rc = np.abs(a / wa - 1) / U, np.abs(c / wc - 1) / U
    print(f"    a: worst {ra.max():.2f} U, c: worst {rc.max():.2f} U", flush=True)
    assert np.all(ra <= wc * et + 2.01) and np.all(rc <= wa * et + 3.01)


def test_scan_nan_stays_in_its_column():
    for shape in ((3, 100, 1), (1, 100, 3)):
        g = torch.zeros(shape, device="cuda")
        u = torch.ones(shape, device="cuda")
        idx = (1, 50, 0) if shape[0] == 3 else (0, 50, 1)
        for t in (g, u):
            t[idx] = float("nan")
            h, last, st = R().wbmm_scan_forward(g, u, 1, h_last=True, states=True)
            bad = torch.isnan(h).reshape(3, 100) if shape[0] == 3 else torch.isnan(h)[0].T
            assert bad[1, 50:].all() and not bad[1, :50].any() and not bad[[0, 2]].any()
            t[idx] = 0.0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("O,L,I", [(3, 1, 5), (4, 100, 1), (3, 900, 1), (2, 9000, 1), (2, 300, 5), (2, 70, 96),
                                   (1, 70000, 2), (1, 70000, 1)])
def test_scan_infinite_values_stay_in_their_column(O, L, I, bf16):
    """From an infinite h0 or u on nothing finite, before it and beside it what there was without it; a
    gradient's infinity runs the other way. Half of the gates forget so fast that products of them
    underflow."""
    g, u, dh, h0, dl = draw((O, L, I), bf16, 12)
    g[:, 1::2] = -25
    dt = torch.bfloat16 if bf16 else torch.float32
    gd, ud, dd, s0, sl = dev(g).to(dt), dev(u).to(dt), dev(dh).to(dt), dev(h0), dev(dl)
    o, i, t = O - 1, I // 2, L // 3
    inf = float("inf")

    def run(u, h0):
        h, last, st = R().wbmm_scan_forward(gd, u, 1, h0=h0, h_last=True, states=True)
        return h, last[:, None], st

    def check(got, want, first):
        for a, b, k in zip(got, want, first):
            mine = a[o, :, i]
            assert torch.equal(mine[:k], b[o, :k, i]) and not torch.isfinite(mine[k:]).any()
            a, b = a.clone(), b.clone()
            a[o, :, i] = b[o, :, i] = 0
            assert torch.equal(a, b)

    want = run(ud, s0)
    bad = s0.clone()
    bad[o, i] = inf
    check(run(ud, bad), want, (0, 0, 0))
    bad = ud.clone()
    bad[o, t, i] = -inf
    check(run(bad, s0), want, (t, 0, t // 32 + 1))

    def back(dh, dl):
        dg, du, d0 = R().wbmm_scan_backward(gd, want[2], dh, 1, u=ud, dh_last=dl)
        return dg.flip(1), du.flip(1), d0[:, None]

    base = back(dd, sl)
    bad = sl.clone()
    bad[o, i] = -inf
    check(back(dd, bad), base, (0, 0, 0))
    bad = dd.clone()
    bad[o, t, i] = inf
    check(back(bad, sl), base, (L - 1 - t, L - 1 - t, 0))


@pytest.mark.parametrize("O,L,I", [(8, 1, 192), (5, 37, 1), (1, 9000, 1), (1, 3000, 4), (4, 70, 3),
                                   (1, 70000, 1), (1, 70000, 2)])
def test_scan_state_updated_in_place(O, L, I):
    g, u, _, h0, _ = draw((O, L, I), False, 6)
    gd, ud = dev(g), dev(u)
    h, last, _ = R().wbmm_scan_forward(gd, ud, 1, h0=dev(h0), h_last=True)
    st = dev(h0)
    h2, st2, _ = R().wbmm_scan_forward(gd, ud, 1, h0=st, h_last=st)
    assert st2.data_ptr() == st.data_ptr() and torch.equal(st, last) and torch.equal(h, h2)


def test_scan_steps_one_by_one_equal_one_run():
    O, L, I = 4, 50, 24
    g, u, _, h0, _ = draw((O, L, I), False, 9)
    h, last, _ = R().wbmm_scan_forward(dev(g), dev(u), 1, h0=dev(h0), h_last=True)
    st = dev(h0)
    for t in range(L):
        ht, st, _ = R().wbmm_scan_forward(dev(g[:, t:t + 1]), dev(u[:, t:t + 1]), 1, h0=st, h_last=st)
        assert torch.allclose(ht[:, 0], h[:, t], rtol=0, atol=60 * 2.0 ** -22)
    assert torch.allclose(st, last, rtol=0, atol=60 * 2.0 ** -22)


@pytest.mark.parametrize("dim", [0, 1, 2, 3, -1])
def test_scan_any_dimension(dim):
    shape = (3, 5, 14, 9)
    rng = np.random.default_rng(0)
    g, u = (rng.standard_normal(shape).astype(np.float32) for _ in range(2))
    h, last, st = R().wbmm_scan_forward(dev(g), dev(u), dim, h_last=True, states=True)
    mv = lambda a: np.moveaxis(a, dim, -1).reshape(-1, shape[dim], 1).astype(np.float64)
    wh, wl, _, bh, bl, _ = Q.scan_forward(mv(g), mv(u))
    close(torch.movedim(h, dim, -1).contiguous(), wh, bh, False, "h")
    close(last, wl, bl, False, "h_last")
    assert st.shape[dim] == 1


@pytest.mark.parametrize("O,L,I,bf16", [(3, 130, 1, False), (2, 70, 5, True), (3, 77, 4, True),
                                        (1, 9000, 1, True), (1, 3000, 3, False), (4, 1, 9, True),
                                        (1, 70000, 1, False), (1, 66000, 2, True)])
def test_scan_writes_only_its_outputs(O, L, I, bf16):
    dt = torch.bfloat16 if bf16 else torch.float32
    g, u, dh, h0, dl = draw((O, L, I), bf16, 5)
    N, G = O * L * I, 67    # odd guard: outputs at the element's own alignment

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * G,), 33.0, dtype=dtype, device="cuda")
        return buf, buf[G:G + n].view(shape)

    def intact(buf):
        b = buf.float().cpu().numpy()
        return np.all(b[:G] == 33) and np.all(b[-G:] == 33)

    ck = -(-L // 32)
    bh, h = guarded((O, L, I), dt)
    bl, last = guarded((O, I), torch.float32)
    bs, st = guarded((O, ck, I), torch.float32)
    need = max(R().wbmm_scan_forward_workspace_bytes(O, L, I),
               R().wbmm_scan_backward_workspace_bytes(O, L, I, False))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    gd, ud, dd = (dev(a).to(dt) for a in (g, u, dh))
    wsp = ws[:need] if need else None
    lens = dev(np.array([max(L - 40, 1)], np.int32))
    for ln in (None, lens):
        h.fill_(float("nan")), st.fill_(float("nan"))
        R().wbmm_scan_forward(gd, ud, 1, h0=dev(h0), h=h, h_last=last, states=st, lens=ln, workspace=wsp)
        assert torch.isfinite(h.float()).all() and torch.isfinite(st).all()
        bg, dg = guarded((O, L, I), dt)
        bu, du = guarded((O, L, I), dt)
        b0, d0 = guarded((O, I), torch.float32)
        dg.fill_(float("nan")), du.fill_(float("nan"))
        R().wbmm_scan_backward(gd, st, dd, 1, u=ud, dg=dg, du=du, dh0=d0, lens=ln, workspace=wsp)
        assert torch.isfinite(dg.float()).all() and torch.isfinite(du.float()).all()
        kept = [t.clone() for t in (dg, du, d0)]
        R().wbmm_scan_backward(gd, None, dd, 1, u=ud, h0=dev(h0), dg=dg, du=du, dh0=d0, lens=ln,
                               workspace=wsp)
        # the states are joined in another order here: either side is within the oracle's bound
        # and half a step of the exact value, so they differ by twice that at most
        n = None if ln is None else np.full(O, max(L - 40, 1))
        f = [v.astype(np.float64) for v in (g, u, h0, dh)]
        want = Q.scan_backward(*f, n=n, bf16=bf16)
        half = [2.0 ** -8 if bf16 else 2.0 ** -24] * 2 + [2.0 ** -24]
        for p, q, w, b, e in zip(kept, (dg, du, d0), want[:3], want[3:], half):
            diff = (p.double() - q.double()).abs().cpu().numpy()
            assert np.all(diff <= 2 * (b * (1 + e) + e * np.abs(w) + 1e-36))
        for b in (bh, bl, bs, bg, bu, b0):
            assert intact(b)
        assert torch.all(ws[need:] == 77)


def test_scan_stream_and_graph():
    for shape in ((6, 300, 1), (2, 100, 20), (1, 9000, 2), (1, 70000, 2), (1, 70000, 1)):
        g, u, dh, h0, dl = (dev(a) for a in draw(shape, False, 1))

        def both(stream=None):
            h, last, st = R().wbmm_scan_forward(g, u, 1, h0=h0, h_last=True, states=True, stream=stream)
            return [h, last, st, *R().wbmm_scan_backward(g, st, dh, 1, u=u, dh_last=dl, stream=stream)]

        want = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = both(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both()
        for k in range(3):
            for t in out:
                t.fill_(float(k))
            both()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_scan_binding_refusals():
    M = R()
    g = torch.zeros(2, 40, 3, device="cuda")
    st = torch.zeros(2, 2, 3, device="cuda")
    h0 = torch.zeros(2, 3, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    bad = [
        lambda: M.wbmm_scan_forward(g, g.bfloat16(), 1), lambda: M.wbmm_scan_forward(g, g[:1], 1),
        lambda: M.wbmm_scan_forward(g, g, 3), lambda: M.wbmm_scan_forward(g.cpu(), g, 1),
        lambda: M.wbmm_scan_forward(g.half(), g.half(), 1), lambda: M.wbmm_scan_forward(g[:0], g[:0], 1),
        lambda: M.wbmm_scan_forward(g, g, 1, h0=h0[:1]), lambda: M.wbmm_scan_forward(g, g, 1, h=g),
        lambda: M.wbmm_scan_forward(g, g, 1, lens=i32(1, 2, 3)),
        lambda: M.wbmm_scan_forward(g, g, 1, lens=i32()),
        lambda: M.wbmm_scan_forward(g, g, 1, lens=torch.tensor([1, 2], device="cuda")),
        lambda: M.wbmm_scan_forward(g.transpose(0, 1), g.transpose(0, 1), 1),
        lambda: M.wbmm_scan_backward(g, st, g, 1), lambda: M.wbmm_scan_backward(g, st[:, :1], g, 1, u=g),
        lambda: M.wbmm_scan_backward(g, st, g, 1, u=g, u_ckpt=(g, g)),
        lambda: M.wbmm_scan_backward(g, st, g, 1, u=g, dg=g),
        lambda: M.wbmm_scan_backward(g, st, g, 1, u_ckpt=M.wbmm_ckpt_pack(g), fmt="x"),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(M.WbmmError):
            f()
            pytest.fail(f"call {k} was accepted")
