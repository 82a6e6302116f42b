"""The block oracle against other ways of computing the same (CPU)."""
import numpy as np
import pytest

from oracle import block_oracle as K
from oracle import ops_oracle as Q

rng = np.random.default_rng(3)


def _fd(f, x, d, h=1e-6):
    """Central difference of the scalar f along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("with_res,with_w", [(True, True), (False, True), (True, False)])
def test_norm_backward_by_differences(with_res, with_w):
    x, dy, ds = (rng.standard_normal((3, 5, 4)) for _ in range(3))
    res = rng.standard_normal((3, 5, 4)) if with_res else None
    w = rng.standard_normal(5) if with_w else None

    def loss(x_, w_):
        t, y = K.norm_forward(x_, res, w_, 1e-3)
        return (y * dy).sum() + (t * ds).sum()

    t, _ = K.norm_forward(x, res, w, 1e-3)
    dx, dw, _, _ = K.norm_backward(t, dy, ds, w, 1e-3)
    d = rng.standard_normal(x.shape)
    assert np.isclose(_fd(lambda z: loss(z, w), x, d), (dx * d).sum(), rtol=1e-6)
    if with_w:
        d = rng.standard_normal(5)
        assert np.isclose(_fd(lambda z: loss(x, z), w, d), (dw * d).sum(), rtol=1e-6)


def test_norm_of_torch():
    torch = pytest.importorskip("torch")
    x, w = rng.standard_normal((2, 7, 3)), rng.standard_normal(7)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x).permute(0, 2, 1), (7,),
                                        torch.from_numpy(w), eps=1e-5).permute(0, 2, 1).numpy()
    assert np.allclose(K.norm_forward(x, None, w, 1e-5)[1], want, rtol=1e-12)


def test_philox_of_the_paper():
    """A published known answer of Philox 4x32 with 7 rounds: counter and key zero."""
    z = K.philox([0], 0, 0, 0)[0]
    assert [int(x) for x in z] == [0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48]


def test_adamw_against_torch():
    torch = pytest.importorskip("torch")
    p = rng.standard_normal(50)
    t = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    m = v = np.zeros(50)
    p32, m32, v32 = p.astype(np.float32), np.zeros(50, np.float32), np.zeros(50, np.float32)
    kw = dict(lr=1e-2, b1=0.9, b2=0.99, eps=1e-6, wd=0.1)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        t.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = K.adamw64(p, g, m, v, step=step, **kw)
        p32, m32, v32 = K.adamw(p32, g.astype(np.float32), m32, v32, step=step, **kw)
        assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)
    assert np.abs(p32 - p).max() < 1e-6


def test_dither_neighbours_and_mean():
    """A code is one of the two neighbours of its value, and the mean over many draws is the value: a draw
    is a step (up to 2^-3 of the value) times a coin, so that over 4000 the mean is within 6 standard
    deviations, 6 * 2^-4 / sqrt(4000) of the value."""
    x = (rng.standard_normal(32) * np.exp(rng.standard_normal(32) * 2)).astype(np.float32)
    sums, grid = np.zeros(32), np.sort(Q.code_values("e4m3")[:127])
    for s in range(4000):
        u = rng.integers(0, 1 << 16, 32).astype(np.float32) * np.float32(2.0 ** -16)
        c, sc = K._dither(x, u, False)
        val = Q.unpack(c, sc, "e4m3")
        f = Q.factor(sc[0])
        up = grid[np.minimum(np.searchsorted(grid, np.abs(x) / f), 126)] * f
        down = grid[np.searchsorted(grid, np.abs(x) / f, side="right") - 1] * f
        assert np.all((np.abs(val) == up) | (np.abs(val) == down))
        sums += val
    step = np.maximum(np.abs(x) * 2.0 ** -3, 2.0 ** -9 * f)
    assert np.all(np.abs(sums / 4000 - x) <= 6 * 0.5 * step / np.sqrt(4000) + 2.0 ** -16 * step)


def test_dither_keeps_a_root_above_zero():
    x = np.zeros(32, np.float32)
    x[0], x[1] = 1.0, 1e-12
    c, sc = K._dither(x, np.zeros(32, np.float32), True)
    assert c[1] == 1 and np.all(c[2:] == 0)


def _delta_inputs(B=2, L=5, Hk=1, H=2, dk=3, dv=2):
    f = rng.standard_normal
    return dict(q=f((B, L, Hk, dk)), k=f((B, L, Hk, dk)) * 0.5, v=f((B, L, H, dv)), g=f((B, L, H)) + 1,
                beta=f((B, L, H)), s0=f((B, H, dk, dv)))


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", [None, [3, 0]])
def test_delta_backward_by_differences(reverse, lens):
    x = _delta_inputs()
    do, dl = rng.standard_normal((2, 5, 2, 2)), rng.standard_normal((2, 2, 3, 2))

    def loss(**kw):
        o, last, _, _ = K.delta_forward(**{**x, **kw}, lens=lens, reverse=reverse, scale=0.7)
        return (o * do).sum() + (last * dl).sum()

    grads = K.delta_backward(**x, do=do, ds_last=dl, lens=lens, reverse=reverse, scale=0.7)
    for name, gr in zip(("q", "k", "v", "g", "beta", "s0"), grads):
        d = rng.standard_normal(gr.shape)
        assert np.isclose(_fd(lambda z: loss(**{name: z}), x[name], d), (gr * d).sum(), rtol=1e-6,
                          atol=1e-9), name


def test_delta_overwrites_a_key():
    """b near 1 and a key of length 1: what was stored under it is replaced."""
    one = np.zeros((1, 2, 1, 2))
    one[..., 0] = 1
    v = np.array([[[[3.0]], [[5.0]]]])
    big = np.full((1, 2, 1), 40.0)
    o, last, _, _ = K.delta_forward(one, one, v, big, big, None, None, False, 1.0)
    assert np.allclose(o[0, :, 0, 0], [3, 5]) and np.allclose(last[0, 0, :, 0], [5, 0])


def _delta_case(B, L, Hk, H, dk, dv, gate):
    mk = lambda *s: rng.standard_normal(s)  # noqa: E731
    unit = lambda t: t / np.linalg.norm(t, axis=-1, keepdims=True)  # noqa: E731
    return ([unit(mk(B, L, Hk, dk)), unit(mk(B, L, Hk, dk)), mk(B, L, H, dv), 1.5 * mk(B, L, H) + gate, mk(B, L, H)],
            0.3 * mk(B, H, dk, dv), mk(B, L, H, dv), mk(B, H, dk, dv), None, False, dk ** -0.5)


def test_the_bounds_of_the_gates_gradients_see_mistakes():
    """The bounds that the GPU tests hold dg and dbeta to: zeros, a wrong sign, 2 % too little and a missing <S_C, D>
    are outside of them in some head at every size and gate. dg itself is below fp32's roundings of what it is
    summed from where a gate lets nothing pass (-100); there only what is missing shows."""
    pytest.importorskip("torch")
    from tests.test_gpu_delta import GATES, gate_bounds
    n = lambda t: np.sqrt((t * t).sum(1))  # noqa: E731
    for size, gate in GATES:
        args = _delta_case(*size, gate)
        want = K.delta_backward(*args[0], *args[1:])[3:5]
        _, _, last = K.delta_gate_bounds(*args[0], *args[1:])
        for h in (2.0 ** -24, 2.0 ** -8):
            tol = gate_bounds(*args, want, h)
            for w, t in zip(want, tol):
                if gate > -100 or w is want[1]:
                    for wrong in (0 * w, -w) + ((w * 0.98,) if gate < 100 else ()):      # there subnormal
                        assert (n(wrong - w) > t).any(), (size, gate, h)
            assert (n(last) > tol[0]).any(), (size, gate, h)


@pytest.mark.parametrize("lens,reverse", [(None, False), ([70, 3], True)])
def test_the_gates_gradients_from_their_terms(lens, reverse):
    """d log y_i = q.dq + k.row - k.col, summed from t to the chunk's end, and <S_C, D>: the identity that the bounds
    (and the kernels) rest on, against the step-by-step gradient."""
    args = list(_delta_case(2, 70, 1, 2, 8, 5, 1.0))
    args[4], args[5] = lens, reverse
    (q, k, v, g, be), s0, do, dl, _, _, scale = args
    w = K.delta_backward(*args[0], *args[1:])
    _, _, last = K.delta_gate_bounds(*args[0], *args[1:])
    for i in range(2):
        order = K._seq(70, 70 if lens is None else lens[i], reverse)
        for h in range(2):
            a, b = 1 / (1 + np.exp(-g[i, :, h])), 1 / (1 + np.exp(-be[i, :, h]))
            run, D = [s0[i, h]], dl[i, h]
            for p in order:
                A = a[p] * run[-1]
                run.append(A + b[p] * np.outer(k[i, p, 0], v[i, p, h] - k[i, p, 0] @ A))
            tail = 0.0
            for t in range(len(order) - 1, -1, -1):
                p, kk, qq = order[t], k[i, order[t], 0], q[i, order[t], 0]
                if t == len(order) - 1 or (t + 1) % K.CHUNK == 0:
                    tail = (run[t + 1] * D).sum()
                    assert np.isclose((1 - a[p]) * tail, last[i, p, h])
                G = scale * do[i, p, h]
                D = D + np.outer(qq, G)
                A, Dk = a[p] * run[t], kk @ D
                row, col = -b[p] * (A @ Dk), b[p] * (D @ (v[i, p, h] - kk @ A))
                tail += qq @ (run[t + 1] @ G) + kk @ row - kk @ col
                assert np.isclose((1 - a[p]) * tail, w[3][i, p, h], atol=1e-12)
                D = a[p] * (D - b[p] * np.outer(kk, Dk))
