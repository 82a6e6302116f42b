"""Pins of the checkpoint and recurrence oracles (CPU, no HIP code)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import ops_oracle as Q


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_code_values_are_the_formats(fmt):
    b = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = b.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.code_values(fmt), want, equal_nan=True)


@pytest.mark.parametrize("fmt,step", [("int8", 0.5 / 63.5), ("e4m3", 2.0 ** -4)])
def test_pack_is_off_by_half_a_step(fmt, step):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal(1000) * np.exp(rng.standard_normal(1000) * 3)).astype(np.float32)
    codes, scales = Q.pack(x, fmt)
    v = Q.unpack(codes, scales, fmt)
    x = x.astype(np.float64)
    for k in range(0, 1000, 32):
        xs, vs = x[k:k + 32], v[k:k + 32]
        if fmt == "int8":   # half a step of at most amax / 63.5
            assert np.abs(xs - vs).max() <= step * np.abs(xs).max()
        else:               # relative, down to the format's least step
            least = 2.0 ** (int(scales[k // 32]) - 127 - 10)
            assert np.all(np.abs(xs - vs) <= np.maximum(step * np.abs(xs), least))


@pytest.mark.parametrize("fmt,top", [("int8", 127), ("e4m3", 448)])
def test_pack_scale_borders(fmt, top):
    """The largest value just at, and just above, what an exponent holds."""
    x = np.zeros(96, np.float32)
    x[0], x[32], x[64] = top, np.nextafter(np.float32(top), np.float32(1e9)), 0
    codes, scales = Q.pack(x, fmt)
    assert list(scales) == [127, 128, 1]
    assert Q.unpack(codes, scales, fmt)[0] == top


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_matches_a_scalar_loop(reverse):
    rng = np.random.default_rng(1)
    g, u, h0 = rng.standard_normal((3, 9, 2)), rng.standard_normal((3, 9, 2)), rng.standard_normal((3, 2))
    n = [9, 0, 5]
    h, last, states = Q.scan_forward(g, u, h0, n, reverse)[:3]
    for o in range(3):
        for i in range(2):
            v = h0[o, i]
            seq = range(n[o])[::-1] if reverse else range(n[o])
            for t in seq:
                a = 1 / (1 + np.exp(-g[o, t, i]))
                v = a * v + (1 - a) * u[o, t, i]
                assert abs(h[o, t, i] - v) < 1e-12
            assert abs(last[o, i] - v) < 1e-12 and states[o, 0, i] == h0[o, i]
        assert np.all(h[o, n[o]:] == 0)


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_backward_by_differences(reverse):
    rng = np.random.default_rng(2)
    shape = (2, 7, 3)
    g, u, dh = (rng.standard_normal(shape) for _ in range(3))
    h0, dl = rng.standard_normal((2, 3)), rng.standard_normal((2, 3))
    n = [7, 4]

    def loss(g, u, h0):
        h, last = Q.scan_forward(g, u, h0, n, reverse)[:2]
        return np.sum(h * dh) + np.sum(last * dl)

    dg, du, d0 = Q.scan_backward(g, u, h0, dh, dl, n, reverse)[:3]
    eps = 1e-5
    for arr, grad, at in ((g, dg, 0), (u, du, 1), (h0, d0, 2)):
        for idx in np.ndindex(arr.shape):
            lo, hi = arr.copy(), arr.copy()
            lo[idx] -= eps
            hi[idx] += eps
            args = [g, u, h0]
            args[at] = hi
            up = loss(*args)
            args[at] = lo
            assert abs((up - loss(*args)) / (2 * eps) - grad[idx]) < 1e-8, (at, idx)
