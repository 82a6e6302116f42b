"""CPU oracle in numpy for the RMS norm, the AdamW step and the gated delta rule. It shares nothing with
the HIP path. The norm and the delta rule are fp64, step by step, each result beside the magnitudes that
a bound on fp32 arithmetic is formed from; AdamW is defined operation by operation, so its oracle is
fp32 in the same order, and fp64 beside it."""
import numpy as np

from oracle import ops_oracle as Q

U = 2.0 ** -24            # half a step of fp32
GROUP, CHUNK = 32, 64


# --------------------------------------------------------------------------------- RMS norm
def norm_forward(x, res, w, eps):
    """x: (outer, len, inner) fp64. Returns t and y."""
    t = x if res is None else x + res
    y = t / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps)
    return t, y if w is None else y * w[None, :, None]


def norm_backward(s, dy, ds, w, eps):
    """dx, dw and the magnitudes that their errors are proportional to."""
    r = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    h = s * r
    g = dy if w is None else dy * w[None, :, None]
    dx = r * (g - h * np.mean(g * h, axis=1, keepdims=True))
    mag = r * (np.abs(g) + np.abs(h) * np.mean(np.abs(g * h), axis=1, keepdims=True))
    if ds is not None:
        dx, mag = dx + ds, mag + np.abs(ds)
    return dx, np.sum(dy * h, axis=(0, 2)), mag, np.sum(np.abs(dy * h), axis=(0, 2))


# --------------------------------------------------------------------------------- AdamW
def philox(index4, tensor, step, seed, rounds=7):
    """(n, 4) words of Philox 4x32 for the counters (index4, tensor, step)."""
    m32 = np.uint64(0xffffffff)
    i = np.asarray(index4, np.uint64)
    c = [i & m32, i >> np.uint64(32), np.full(i.shape, tensor, np.uint64),
         np.full(i.shape, step, np.uint64)]
    k0, k1 = seed & 0xffffffff, (seed >> 32) & 0xffffffff
    for _ in range(rounds):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & m32,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return np.stack(c, -1)


def _dither(x, u, keep):
    """codes and scales of fp32 values x, u in [0, 1) deciding between the neighbouring codes."""
    n = x.size
    pad = -n % GROUP
    v = np.concatenate([x, np.zeros(pad, np.float32)]).reshape(-1, GROUP)
    u = np.concatenate([u, np.zeros(pad, np.float32)]).reshape(-1, GROUP)
    codes, scales = np.zeros(v.shape, np.uint8), np.zeros(v.shape[0], np.uint8)
    vals = Q.code_values("e4m3")
    code_of = {float(vals[c]): c for c in range(127)}
    for g in range(v.shape[0]):
        if not np.all(np.isfinite(v[g])):
            scales[g] = 255
            continue
        amax, e = float(np.abs(v[g]).max()), -126
        if amax > 0:
            e = max(-126, int(np.floor(np.log2(amax))) - 10)
        while amax > 448.0 * 2.0 ** e:
            e += 1
        while e > -126 and amax <= 448.0 * 2.0 ** (e - 1):
            e -= 1
        scales[g] = e + 127
        for j in range(GROUP):
            q = float(v[g, j]) * 2.0 ** -e
            mag = abs(q)
            b = (max(-6, int(np.floor(np.log2(mag)))) if mag else -6) - 3
            k = np.floor(np.float32(np.float32(mag * 2.0 ** -b) + u[g, j]))
            if keep and mag > 0 and k < 1:
                k = 1.0
            codes[g, j] = code_of[float(k) * 2.0 ** b] | (0x80 if np.signbit(q) else 0)
    return codes.reshape(-1)[:n], scales


def adamw(p, g, m, v, *, lr, b1, b2, eps, wd, step, tensor=0, seed=0, lr_factor=None,
          grad_factor=None, first=0):
    """One tensor's step in fp32, operation by operation. m, v: fp32 arrays, or (codes, scales) of m
    and of v's root. first: the index of the arrays' first element in its tensor (a multiple of 32). Returns p, m, v
    in the same forms."""
    f = np.float32
    lr = lr * float(lr_factor) if lr_factor is not None else lr
    k1, k2 = f(lr / (1 - b1 ** step)), f(1 / np.sqrt(1 - b2 ** step))
    keep = f(1 - lr * wd)
    g = (g.astype(f) * f(1 if grad_factor is None else grad_factor)).astype(f)
    small = isinstance(m, tuple)
    if small:
        mm = Q.unpack(m[0], m[1], "e4m3").astype(f)
        r = Q.unpack(v[0], v[1], "e4m3").astype(f)
        vv = r * r
    else:
        mm, vv = m, v
    with np.errstate(all="ignore"):
        mm = f(b1) * mm + f(1 - b1) * g
        vv = f(b2) * vv + f(1 - b2) * (g * g)
        root = np.sqrt(vv)
        p = p * keep - k1 * mm / (root * k2 + f(eps))
    assert p.dtype == f and mm.dtype == f
    if not small:
        return p, mm, vv
    n = p.size
    words = philox(first // 4 + np.arange(-(-n // 4)), tensor, step, seed).reshape(-1)[:n]
    um = (words & np.uint64(0xffff)).astype(f) * f(2.0 ** -16)
    ur = (words >> np.uint64(16)).astype(f) * f(2.0 ** -16)
    return p, _dither(mm, um, False), _dither(root, ur, True)


def adamw64(p, g, m, v, *, lr, b1, b2, eps, wd, step):
    """The same in fp64, states not rounded."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * wd * p - lr * mh / (np.sqrt(vh) + eps), m, v


# --------------------------------------------------------------------------------- delta rule
def _sig(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def _seq(L, n, reverse):
    n = min(max(int(n), 0), L)
    return [n - 1 - t if reverse else t for t in range(n)]


def delta_forward(q, k, v, g, beta, s0, lens, reverse, scale):
    """All fp64: q, k (B, L, Hk, dk), v (B, L, H, dv), g, beta (B, L, H). Returns o, the last state, the
    states every 64 steps, and the largest norm of a column of S or entry of v, per head."""
    B, L, H, dv = v.shape
    Hk, dk = q.shape[2:]
    nch = -(-L // CHUNK)
    o, last = np.zeros((B, L, H, dv)), np.zeros((B, H, dk, dv))
    states, M = np.zeros((B, H, nch, dk, dv)), np.zeros((B, H))
    a, b = _sig(np.clip(g, -87, 87)), _sig(beta)
    for i in range(B):
        order = _seq(L, L if lens is None else lens[i], reverse)
        for h in range(H):
            hk = h // (H // Hk)
            S = np.zeros((dk, dv)) if s0 is None else s0[i, h].copy()
            top = np.sqrt((S * S).sum(0)).max()
            for t, p in enumerate(order):
                if t % CHUNK == 0:
                    states[i, h, t // CHUNK] = S
                kk = k[i, p, hk]
                S = a[i, p, h] * S
                S = S + b[i, p, h] * np.outer(kk, v[i, p, h] - kk @ S)
                o[i, p, h] = scale * (q[i, p, hk] @ S)
                top = max(top, np.sqrt((S * S).sum(0)).max(), np.abs(v[i, p, h]).max())
            for c in range(-(-len(order) // CHUNK), nch):
                states[i, h, c] = S
            last[i, h], M[i, h] = S, top
    return o, last, states, M


def delta_backward(q, k, v, g, beta, s0, do, ds_last, lens, reverse, scale):
    """dq, dk, dv, dg, dbeta, ds0; then per head the largest norm of a column of D or of scale |q| do, and
    per step the magnitudes of the dot products that dg's sums over a chunk are made of."""
    B, L, H, dv_ = v.shape
    Hk, dk_ = q.shape[2:]
    a, b = _sig(np.clip(g, -87, 87)), _sig(beta)
    na, nb = _sig(-np.clip(g, -87, 87)), _sig(-beta)       # 1 - a and 1 - b, where a and b are 1 in fp64 too
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, dbe, ds0 = np.zeros_like(g), np.zeros_like(beta), np.zeros((B, H, dk_, dv_))
    MD, dots = np.zeros((B, H)), np.zeros_like(g)
    for i in range(B):
        order = _seq(L, L if lens is None else lens[i], reverse)
        for h in range(H):
            hk = h // (H // Hk)
            S = np.zeros((dk_, dv_)) if s0 is None else s0[i, h].copy()
            run = [S]
            for p in order:
                kk, A = k[i, p, hk], a[i, p, h] * run[-1]
                run.append(A + b[i, p, h] * np.outer(kk, v[i, p, h] - kk @ A))
            D = np.zeros((dk_, dv_)) if ds_last is None else ds_last[i, h].copy()
            top = np.sqrt((D * D).sum(0)).max()
            mags = np.zeros(len(order))
            for t in range(len(order) - 1, -1, -1):
                p = order[t]
                S0, S1 = run[t], run[t + 1]
                qq, kk, bb, aa = q[i, p, hk], k[i, p, hk], b[i, p, h], a[i, p, h]
                G = scale * do[i, p, h]
                D = D + np.outer(qq, G)
                top = max(top, np.sqrt((D * D).sum(0)).max(), np.abs(G).max() * np.linalg.norm(qq))
                A = aa * S0
                err, Dk = v[i, p, h] - kk @ A, kk @ D
                tq, row, col = S1 @ G, -bb * (A @ Dk), bb * (D @ err)
                dq[i, p, hk] += tq
                dk[i, p, hk] += row + col
                dv[i, p, h] = bb * Dk
                dbe[i, p, h] = bb * nb[i, p, h] * (Dk @ err)
                dA = D - bb * np.outer(kk, Dk)
                dg[i, p, h] = na[i, p, h] * (dA * A).sum()
                mags[t] = (np.linalg.norm(qq) * np.linalg.norm(tq) + np.linalg.norm(kk) *
                           (np.linalg.norm(row) + np.linalg.norm(col)))
                D = aa * dA
            # dg of a step is a sum over the steps from it to the end of its chunk, and the product of
            # the state after the chunk with its gradient
            for t, p in enumerate(order):
                e = min((t // CHUNK + 1) * CHUNK, len(order))
                dots[i, p, h] = mags[t // CHUNK * CHUNK: e].sum()
            ds0[i, h], MD[i, h] = D, top
    return dq, dk, dv, dg, dbe, ds0, MD, dots


def delta_gate_bounds(q, k, v, g, beta, s0, do, ds_last, lens, reverse, scale):
    """What dg and dbeta are sums of, in the order that a chunked computation forms them, fp64, (B, L, H) each:
    the size of dg's terms (the dot products of the steps from t to its chunk's end, and of the state after the chunk
    with its gradient, taken as independent), of dbeta's, and that last product's own share of dg."""
    B, L, H, dv = v.shape
    Hk, dk = q.shape[2:]
    a, b = _sig(np.clip(g, -87, 87)), _sig(beta)
    na, nb = _sig(-np.clip(g, -87, 87)), _sig(-beta)
    tg, tb, last = (np.zeros((B, L, H)) for _ in range(3))
    for i in range(B):
        order = _seq(L, L if lens is None else lens[i], reverse)
        for h in range(H):
            hk = h // (H // Hk)
            run = [np.zeros((dk, dv)) if s0 is None else s0[i, h]]
            for p in order:
                kk, A = k[i, p, hk], a[i, p, h] * run[-1]
                run.append(A + b[i, p, h] * np.outer(kk, v[i, p, h] - kk @ A))
            D = np.zeros((dk, dv)) if ds_last is None else ds_last[i, h]
            sq, whole, size = 0.0, 0.0, 0.0
            for t in range(len(order) - 1, -1, -1):
                p, norm = order[t], np.linalg.norm
                if t == len(order) - 1 or (t + 1) % CHUNK == 0:
                    S = run[t + 1]
                    whole, size = (S * D).sum(), 2 * norm(S) * norm(D) / np.sqrt(dk * dv)
                    sq = size ** 2
                qq, kk, bb, A = q[i, p, hk], k[i, p, hk], b[i, p, h], a[i, p, h] * run[t]
                G = scale * do[i, p, h]
                D = D + np.outer(qq, G)
                Dk = kk @ D
                row, col = bb * norm(A @ Dk), bb * norm(D @ (v[i, p, h] - kk @ A))
                sq += (norm(qq) * norm(run[t + 1] @ G) + norm(kk) * (row + col)) ** 2
                tg[i, p, h], last[i, p, h] = na[i, p, h] * np.sqrt(sq), na[i, p, h] * whole
                tb[i, p, h] = nb[i, p, h] * (norm(v[i, p, h]) * bb * norm(Dk) + norm(kk) * row)
                D = a[i, p, h] * (D - bb * np.outer(kk, Dk))
    return tg, tb, last
