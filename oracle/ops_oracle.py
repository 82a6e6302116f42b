"""CPU oracle in numpy fp64 for 8-bit activation checkpoints and the gated linear recurrence. It
shares nothing with the HIP path. Beside each recurrence result stands a bound on what fp32
arithmetic may add to it, carried through the same loop."""
import numpy as np

GROUP = 32
CHUNK = 32


# --------------------------------------------------------------------------------- checkpoints
def code_values(fmt):
    """The 256 code values (e4m3: bias 7, no infinities, NaN at 0x7f and 0xff)."""
    if fmt == "int8":
        return np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)
    out = np.empty(256)
    for b in range(256):
        ex, man = (b >> 3) & 15, b & 7
        v = man * 2.0 ** -9 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        if b & 127 == 127:
            v = np.nan
        out[b] = -v if b & 128 else v
    return out


def factor(byte):
    return np.nan if byte == 255 else 2.0 ** (int(byte) - 127)


def pack(x, fmt):
    """(codes, scales) of the flat fp64 values x, by search over the code values."""
    vals = code_values(fmt)
    order = np.argsort(np.where(np.isnan(vals), np.inf, vals), kind="stable")
    order = order[: np.sum(~np.isnan(vals))]
    grid = vals[order]
    top = 127.0 if fmt == "int8" else 448.0
    flat = np.asarray(x, np.float64).reshape(-1)
    codes = np.zeros(flat.size, np.uint8)
    scales = np.zeros(-(-flat.size // GROUP), np.uint8)
    for k in range(scales.size):
        v = flat[k * GROUP:(k + 1) * GROUP]
        if not np.all(np.isfinite(v)):
            scales[k] = 255
            continue
        amax = np.abs(v).max()
        e = -126
        while amax > top * 2.0 ** e:
            e += 1
        scales[k] = e + 127
        for j, q in enumerate(v * 2.0 ** -e):
            d = np.abs(grid - q)
            near = np.flatnonzero(d == d.min())
            best = near[0]
            for m in near:                      # ties: the even code
                if order[m] % 2 == 0:
                    best = m
            c = order[best]
            if fmt == "e4m3" and vals[c] == 0:  # a zero keeps the sign of what it came from
                c = 0x80 if np.signbit(q) else 0
            codes[k * GROUP + j] = c
    return codes.reshape(np.shape(x)), scales


def unpack(codes, scales, fmt):
    f = np.array([factor(b) for b in range(256)])[scales]
    flat = code_values(fmt)[codes.reshape(-1)]
    return (flat * np.repeat(f, GROUP)[: flat.size]).reshape(codes.shape)


# --------------------------------------------------------------------------------- recurrence
# What fp32 may lose, in half steps U of relative error. t = exp(-g): 2 for the hardware's exp2 (one
# step), 1 for the correction that puts back what the exponent it is given leaves out of g log2(e), and
# for bf16 tensors, where that is up to 4.9e-6 |g|, half its square, 2.1e-4 g^2 (at most 1.6). a = 1 / (1 + t):
# t's error times 1 - a, the sum's rounding and one step of the reciprocal; c = t a: both and a rounding.
U = 2.0 ** -24


def gate_bounds(g, bf16):
    """Relative error bounds of a and c = 1 - a."""
    et = (3 + (2.1e-4 * np.minimum(np.abs(g), 87) ** 2 if bf16 else 0)) * U
    one_minus_a = 1 / (1 + np.exp(g))
    ea = one_minus_a * et + U + 2 * U
    return ea, ea + et + U


def _steps(n, s, reverse, L):
    live = s < n
    pos = np.where(live, (n - 1 - s) if reverse else s, 0)
    return live, pos


def scan_forward(g, u, h0=None, n=None, reverse=False, bf16=False):
    """g, u: (outer, len, inner) fp64. Returns h, h_last, states and the bounds of h and h_last."""
    O, L, I = g.shape
    n = np.full(O, L) if n is None else np.asarray(n)
    h = np.zeros((O, I)) if h0 is None else h0.astype(np.float64)
    a, c = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    ea, ec = gate_bounds(g, bf16)
    out, bound = np.zeros_like(g), np.zeros_like(g)
    states, sbound = [], []
    S, E = np.abs(h), np.zeros_like(h)   # sum of magnitudes; error
    r = np.arange(O)
    for s in range(L):
        if s % CHUNK == 0:
            states.append(h.copy())
            sbound.append(E + 40 * U * S)
        live, p = _steps(n, s, reverse, L)
        m = live[:, None]
        ga, gc, gu = a[r, p], c[r, p], u[r, p]
        nh = ga * h + gc * gu
        # every factor of every term of h is off by ea or ec and by one rounding of its product
        # and one of the sum it enters, whatever the order of joining; the third U of a step is for
        # the joins that come one after another (waves, tiles, parts of the axis): they lie 16 steps
        # or more apart and round a term that passes at most twice, however many there are
        nE = ga * E + ga * S * (ea[r, p] + 3 * U) + gc * np.abs(gu) * (ec[r, p] + 3 * U)
        nS = ga * S + gc * np.abs(gu)
        h, E, S = np.where(m, nh, h), np.where(m, nE, E), np.where(m, nS, S)
        out[r[live], p[live]] = h[live]
        # the joins that come by doubling: 6 within a wave and one to the lane before, twice each
        # for the pieces and for the waves, of two roundings: 28, and the first and last join of a
        # term that passes fewer than 16 steps
        bound[r[live], p[live]] = (E + 40 * U * S)[live]
    return out, h, np.stack(states, 1), bound, E + 40 * U * S, np.stack(sbound, 1)


def scan_backward(g, u, h0, dh, dh_last=None, n=None, reverse=False, bf16=False):
    """dg, du, dh0 and their bounds."""
    O, L, I = g.shape
    n = np.full(O, L) if n is None else np.asarray(n)
    a, c = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    ea, ec = gate_bounds(g, bf16)
    r = np.arange(O)
    h = np.zeros((O, I)) if h0 is None else h0.astype(np.float64)
    S, E = np.abs(h), np.zeros_like(h)
    prev, prevE = np.zeros_like(g), np.zeros_like(g)
    for s in range(L):
        live, p = _steps(n, s, reverse, L)
        m = live[:, None]
        ga, gc, gu = a[r, p], c[r, p], u[r, p]
        prev[r[live], p[live]] = h[live]
        prevE[r[live], p[live]] = (E + 40 * U * S)[live]
        nE = ga * E + ga * S * (ea[r, p] + 3 * U) + gc * np.abs(gu) * (ec[r, p] + 3 * U)
        nS = ga * S + gc * np.abs(gu)
        h, E, S = (np.where(m, ga * h + gc * gu, h), np.where(m, nE, E), np.where(m, nS, S))
    R = np.zeros((O, I)) if dh_last is None else dh_last.astype(np.float64)
    RS, RE = np.abs(R), np.zeros_like(R)
    dg, du, bg, bu = (np.zeros_like(g) for _ in range(4))
    for s in range(L - 1, -1, -1):
        live, p = _steps(n, s, reverse, L)
        m = live[:, None]
        ga, gc, d = a[r, p], c[r, p], dh[r, p]
        G, GS = d + R, np.abs(d) + RS
        GE = RE + 40 * U * GS
        x = prev[r, p] - u[r, p]
        w = ga * gc
        du[r[live], p[live]] = (gc * G)[live]
        dg[r[live], p[live]] = (w * x * G)[live]
        bu[r[live], p[live]] = (gc * (GE + np.abs(G) * (ec[r, p] + 2 * U)))[live]
        bg[r[live], p[live]] = (w * (np.abs(x) * GE + np.abs(G) * (
            prevE[r, p] + np.abs(x) * (ea[r, p] + ec[r, p] + 4 * U))))[live]
        nRE = ga * RE + ga * GS * (ea[r, p] + 3 * U)
        R, RE, RS = np.where(m, ga * G, R), np.where(m, nRE, RE), np.where(m, ga * GS, RS)
    return dg, du, R, bg, bu, RE + 40 * U * RS
