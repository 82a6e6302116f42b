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
