"""Gated delta rule against the fp64 oracle, step by step.

Tolerances. The rule contracts for |k| <= 1: an error of a state's column grows no further, and T's entries
are at most 1. Within a chunk a value passes four products in a row (K S, T X, P U or K^T U, the decays) of
up to 64 or 128 terms, with factors good to 2^-24 and fp32 sums: 256 half steps of fp32 of M, the largest
norm of a column of S (or entry of v). Gradients: of M and M_D, the same of D; dq and dk are sums over dv of
such products, dg sums over a chunk of the dot products whose magnitudes the oracle gives. bf16: what only
reaches an output is taken to 2^-17 of each factor: 64 terms of at most 2 M, each good to 2^-16, at random
8 * 2 * 2^-16 = 2^-12 of M, before the output's own rounding. Taken together, outputs are as good relative
to their own norm. The keys have length 1."""
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


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def half(dt):
    return torch.finfo(dt).eps / 2


def near(name, got, want, tol):
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (name, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5],
                           np.broadcast_to(tol, got.shape)[bad][:5])


class Case:
    def __init__(self, B, L, Hk, H, dk, dv, dt=F32, reverse=False, lens=None, s0=True, seed=1, gate=3.0):
        mk = lambda s, sig, k: torch.from_numpy(synth.normal_f32(s, sig, seed + k)).cuda()  # noqa: E731
        unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
        self.dt, self.reverse, self.dk = dt, reverse, dk
        self.q, self.k = unit(mk((B, L, Hk, dk), 1.0, 0)), unit(mk((B, L, Hk, dk), 1.0, 1))
        self.v, self.g = mk((B, L, H, dv), 1.0, 2).to(dt), (mk((B, L, H), 1.5, 3) + gate).to(dt)
        self.beta = mk((B, L, H), 1.0, 4).to(dt)
        self.s0 = mk((B, H, dk, dv), 0.3, 5) if s0 else None
        self.do, self.dl = mk((B, L, H, dv), 1.0, 6).to(dt), mk((B, H, dk, dv), 1.0, 7)
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.hl = lens

    def inputs(self):
        return self.q, self.k, self.v, self.g, self.beta

    def forward(self, **kw):
        return R().wbmm_delta_forward(*self.inputs(), s0=self.s0, lens=self.lens, reverse=self.reverse,
                                      **{"s_last": True, "states": True, **kw})

    def backward(self, states, **kw):
        return R().wbmm_delta_backward(*self.inputs(), self.do, states=states,
                                       s0=self.s0 if states is None else None, ds_last=self.dl, lens=self.lens,
                                       reverse=self.reverse, **kw)

    def check_forward(self, o, last, states):
        x = [f64(t) for t in self.inputs()]
        self.want = K.delta_forward(*x, f64(self.s0), self.hl, self.reverse, self.dk ** -0.5)
        wo, wl, ws, M = self.want
        h, more = half(self.dt), 2.0 ** -12 if self.dt == BF16 else 0.0
        scale = self.dk ** -0.5 * 1.01
        near("o", f64(o), wo, (256 * U + more) * M[:, None, :, None] * scale * (1 + h) + h * np.abs(wo))
        near("s_last", f64(last), wl, 256 * U * M[:, :, None, None] + U * np.abs(wl))
        assert np.linalg.norm(f64(o) - wo) <= (256 * U + more + h) * np.linalg.norm(wo)
        near("states", f64(states), ws, 256 * U * M[:, :, None, None, None] + U * np.abs(ws))

    def check_backward(self, grads):
        x = [f64(t) for t in self.inputs()]
        M = self.want[3]
        scale = self.dk ** -0.5 * 1.01
        *w, MD, dots = K.delta_backward(*x, f64(self.s0), f64(self.do), f64(self.dl), self.hl, self.reverse,
                                        self.dk ** -0.5)
        h, more = half(self.dt), 2.0 ** -12 if self.dt == BF16 else 0.0
        e = (256 * U + more) * (1 + h)
        B, L, Hk, _ = self.q.shape
        H = self.v.shape[2]
        group = lambda t: t.reshape(*t.shape[:-1], Hk, H // Hk).sum(-1)  # noqa: E731
        do1 = np.abs(f64(self.do)).sum(-1)                            # (B, L, H)
        dv1 = self.v.shape[3]
        bound = {"dq": group(scale * M[:, None] * do1)[..., None],
                 "dk": group(np.broadcast_to(3 * dv1 * (M * MD)[:, None], (B, L, H)))[..., None],
                 "dv": MD[:, None, :, None] * np.ones((B, L, 1, 1)),
                 "dg": dots + 3 * dv1 * (M * MD)[:, None], "dbeta": np.broadcast_to(dv1 * (M * MD)[:, None], (B, L, H)),
                 "ds0": MD[:, :, None, None]}
        for (name, m), got, want in zip(bound.items(), grads, w):
            tol = 256 * U * m if name == "ds0" else e * m + h * np.abs(want)
            near(name, f64(got), want, tol + U * np.abs(want))
            if name not in ("dg", "dbeta"):           # differences of larger sums
                # what is below the least normal number 2^-126 of fp32 has steps of its own, or is 0 to a matrix
                # product: each element may be off by that much whatever its value (a gate of -100 gives such)
                most = (e + (0 if name == "ds0" else h)) * np.linalg.norm(want) + 2.0 ** -126 * want.size ** 0.5
                assert np.linalg.norm(f64(got) - want) <= most, name


SIZES = [
    # B, L, Hk, H, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 1, 1, 2, 64, 64), (2, 5, 2, 4, 24, 20), (1, 8, 1, 1, 128, 128), (2, 9, 1, 3, 16, 16),
    (1, 63, 1, 1, 32, 32), (2, 64, 1, 1, 33, 17), (1, 65, 2, 2, 64, 48), (1, 128, 1, 1, 100, 96),
    (3, 129, 1, 2, 48, 40), (1, 200, 1, 1, 128, 128), (2, 130, 3, 3, 65, 77), (1, 300, 2, 6, 8, 5),
    (1, 70, 1, 1, 3, 1), (1, 257, 1, 1, 1, 33), (2, 66, 1, 9, 40, 33),
]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,L,Hk,H,dk,dv", SIZES)
def test_forward_and_backward(B, L, Hk, H, dk, dv, dt):
    print(f"\n[case] delta {B}x{L} heads {Hk}/{H} {dk}x{dv} {dt}", flush=True)
    c = Case(B, L, Hk, H, dk, dv, dt)
    o, last, states = c.forward()
    c.check_forward(o, last, states)
    c.check_backward(c.backward(states))


LENS = [(4, 70, [70, 0, 1, 33]), (3, 130, [64, 129, -5]), (3, 200, [65, 1000, 128]), (2, 7, [0, 6]), (2, 64, [0, 0])]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,L,lens", LENS)
def test_padded_batches(B, L, lens, dt, reverse):
    """What lies past the end is not read: NaN there change nothing."""
    print(f"\n[case] delta padded {B}x{L} {lens} {dt} rev={reverse}", flush=True)
    c = Case(B, L, 2, 4, 24, 20, dt, reverse, lens, seed=11)
    for b, n in enumerate(lens):
        for t in (*c.inputs(), c.do):
            t[b, min(max(n, 0), L):] = float("nan")
    o, last, states = c.forward()
    gr = c.backward(states)
    for b, n in enumerate(lens):
        n = min(max(n, 0), L)
        for t in (o, *gr[:5]):
            assert torch.all(t[b, n:] == 0)
        for t in (*c.inputs(), c.do):
            t[b, n:] = 0
    c.check_forward(o, last, states)
    c.check_backward(gr)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,L,Hk,H,dk,dv", [(2, 130, 1, 2, 64, 48), (1, 200, 1, 1, 128, 128), (1, 5, 1, 1, 16, 16),
                                            (1, 129, 2, 4, 20, 30)])
def test_reversed_and_without_initial_state(B, L, Hk, H, dk, dv, dt):
    c = Case(B, L, Hk, H, dk, dv, dt, reverse=True, s0=False, seed=21)
    out = c.forward()
    c.check_forward(*out)
    c.check_backward(c.backward(out[2]))


@pytest.mark.parametrize("gate", [-100.0, -6.0, 0.0, 12.0, 100.0])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gates_from_nothing_to_everything(gate, dt):
    c = Case(2, 150, 1, 2, 32, 24, dt, gate=gate, seed=31)
    c.g[0, 70], c.g[1, 3], c.g[0, 71] = -200.0, 200.0, float("-inf")
    c.beta[0, 10], c.beta[1, 20], c.beta[0, 30] = 50.0, -50.0, float("inf")
    out = c.forward()
    c.check_forward(*out)
    c.check_backward(c.backward(out[2]))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_the_same_key_again_and_again(dt):
    """A's entries as large as they get: one key, b near 1, nothing forgotten."""
    c = Case(1, 192, 1, 1, 16, 16, dt, gate=20.0, seed=41)
    c.k[:] = c.k[:, :1]
    c.beta[:] = 8.0
    out = c.forward()
    c.check_forward(*out)
    c.check_backward(c.backward(out[2]))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("L,dk,dv", [(150, 64, 48), (64, 128, 128), (9, 24, 20)])
def test_states_formed_again(L, dk, dv, dt):
    """A backward without states equals the one from the forward's, bit for bit."""
    c = Case(2, L, 1, 2, dk, dv, dt, seed=51)
    states = c.forward()[2]
    for a, b in zip(c.backward(states), c.backward(None)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_partial_outputs_and_twice(dt):
    c = Case(2, 150, 2, 4, 64, 48, dt, seed=61)
    o, last, states = c.forward()
    o2, none, none2 = c.forward(s_last=False, states=False)
    assert none is None and none2 is None and torch.equal(o, o2)
    g = c.backward(states)
    h = c.backward(states, ds0=False)
    assert h[5] is None and all(torch.equal(a, b) for a, b in zip(g[:5], h[:5]))
    assert all(torch.equal(a, b) for a, b in zip(g, c.backward(states)))


@pytest.mark.parametrize("L", [1, 8, 100])
def test_state_in_place(L):
    c = Case(2, L, 1, 2, 64, 40, BF16, seed=71)
    o, last, _ = c.forward()
    s = c.s0.clone()
    o2, last2, _ = R().wbmm_delta_forward(*c.inputs(), s0=s, s_last=s)
    assert last2 is s and torch.equal(s, last) and torch.equal(o, o2)
    if L > 8:
        states = c.forward()[2]
        want = c.backward(states)[5]
        d = c.dl.clone()
        R().wbmm_delta_backward(*c.inputs(), c.do, states=states, ds_last=d, ds0=d)
        assert torch.equal(d, want)


def test_single_steps_make_a_sequence():
    """100 calls of one step against one call of 100: two ways of rounding, each within its bound."""
    c = Case(2, 100, 1, 2, 64, 48, BF16, seed=81)
    o, last, states = c.forward()
    c.check_forward(o, last, states)
    s, rows = c.s0.clone(), []
    for t in range(100):
        one = [x[:, t:t + 1].contiguous() for x in c.inputs()]
        rows.append(R().wbmm_delta_forward(*one, s0=s, s_last=s)[0])
    c.check_forward(torch.cat(rows, 1), s, states)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("L,dk,dv", [(130, 64, 48), (5, 64, 48), (70, 128, 128), (100, 20, 12)])
def test_any_alignment(L, dk, dv, dt):
    c = Case(2, L, 1, 2, dk, dv, dt, seed=91)

    def off(t):
        flat = torch.empty(t.numel() + 9, dtype=t.dtype, device="cuda")
        v = flat[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    for n in ("q", "k", "v", "g", "beta", "do", "s0", "dl"):
        setattr(c, n, off(getattr(c, n)))
    out = c.forward(o=off(c.v), s_last=off(c.s0), states=off(torch.empty(2, 2, -(-L // 64), dk, dv, device="cuda")))
    c.check_forward(*out)
    c.check_backward(c.backward(out[2], dq=off(c.q), dk=off(c.k), dv=off(c.v), dg=off(c.g), dbeta=off(c.beta),
                                ds0=off(c.s0)))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("L,dk,dv,lens", [(130, 64, 40, None), (70, 33, 17, [70, 5]), (6, 24, 20, [6, 0]),
                                          (200, 128, 128, [199, 64])])
def test_nothing_else_is_written(L, dk, dv, lens, dt):
    M, pad = R(), 64
    c = Case(2, L, 1, 2, dk, dv, dt, lens=lens, seed=101)
    kept = []

    def guarded(shape, t):
        n = int(np.prod(shape))
        flat = torch.full((n + 2 * pad,), 77 if t == torch.uint8 else 3.0, dtype=t, device="cuda")
        kept.append(flat)
        return flat[pad:pad + n].view(shape)

    st = (2, 2, -(-L // 64), dk, dv)
    sizes = (2, L, 1, 2, dk, dv)
    fw = M.wbmm_delta_forward_workspace_bytes(*sizes, dt)
    bw = M.wbmm_delta_backward_workspace_bytes(*sizes, dt)
    out = c.forward(o=guarded(c.v.shape, dt), s_last=guarded(c.s0.shape, F32), states=guarded(st, F32),
                    workspace=guarded((fw,), torch.uint8) if fw else None)
    gr = c.backward(out[2], dq=guarded(c.q.shape, dt), dk=guarded(c.k.shape, dt), dv=guarded(c.v.shape, dt),
                    dg=guarded(c.g.shape, dt), dbeta=guarded(c.g.shape, dt), ds0=guarded(c.s0.shape, F32),
                    workspace=guarded((bw,), torch.uint8))
    for flat in kept:
        fill = 77 if flat.dtype == torch.uint8 else 3.0
        assert torch.all(flat[:pad] == fill) and torch.all(flat[-pad:] == fill)
    if lens is None:
        c.check_forward(*out)
        c.check_backward(gr)


def test_workspaces_may_hold_anything():
    """NaN in a workspace change nothing."""
    M = R()
    for dt in (F32, BF16):
        c = Case(2, 150, 1, 2, 48, 40, dt, lens=[150, 70], seed=111)
        states = c.forward()[2]
        want = c.backward(states)
        sizes = (2, 150, 1, 2, 48, 40, dt)
        for s in (states, None):
            ws = torch.full((M.wbmm_delta_backward_workspace_bytes(*sizes, s is not None) // 4 + 1,), float("nan"),
                            device="cuda")
            assert all(torch.equal(a, b) for a, b in zip(want, c.backward(s, workspace=ws)))
        ws = torch.full((M.wbmm_delta_forward_workspace_bytes(*sizes) // 4 + 1,), float("nan"), device="cuda")
        assert torch.equal(c.forward(workspace=ws)[2], states)


def test_nan_and_infinities_from_their_chunk_on():
    for dt in (F32, BF16):
        c = Case(1, 200, 1, 2, 32, 24, dt, seed=121)
        o0, l0, s0 = c.forward()
        for name, val in (("k", float("nan")), ("g", float("nan")), ("v", float("inf")), ("beta", float("nan"))):
            x = getattr(c, name)
            keep = x.clone()
            at = (0, 100, 0) if x.dim() == 3 else (0, 100, 0, 3)
            x[at] = val
            o, last, _ = c.forward()
            assert torch.equal(o[:, :64], o0[:, :64])
            hit = o[0, 128:, 0] if name != "v" else o[0, 128:, 0, 3]
            assert hit.isnan().all() or not hit.isfinite().any(), name
            if name == "v":
                rest = [j for j in range(24) if j != 3]
                assert torch.equal(o[..., rest], o0[..., rest])
            if name != "k":      # the key is both heads'
                assert torch.equal(o[:, :, 1], o0[:, :, 1]) or name == "v"
            x.copy_(keep)
        c.q[0, 100, 0, 3] = float("nan")
        o, last, _ = c.forward()
        keep = [t for t in range(200) if t != 100]
        assert o[0, 100].isnan().all() and torch.equal(o[:, keep], o0[:, keep]) and torch.equal(last, l0)


def test_many_heads_and_batches_are_each_their_own():
    """Each sequence of a large batch equals the same sequence alone."""
    for dt, B, L, Hk, H, dk, dv in ((BF16, 70, 100, 2, 4, 64, 64), (F32, 33, 65, 1, 3, 32, 20)):
        c = Case(B, L, Hk, H, dk, dv, dt, seed=131)
        out = c.forward()
        gr = c.backward(out[2])
        for b in (0, B // 2, B - 1):
            one = Case(1, L, Hk, H, dk, dv, dt)
            for n in ("q", "k", "v", "g", "beta", "s0", "do", "dl"):
                setattr(one, n, getattr(c, n)[b:b + 1].contiguous())
            o1 = one.forward()
            assert all(torch.equal(a[b:b + 1], x) for a, x in zip(out, o1))
            assert all(torch.equal(a[b:b + 1], x) for a, x in zip(gr, one.backward(o1[2])))


@pytest.mark.parametrize("dt,B,Hk,H,dk,dv,reverse,s0", [
    (F32, 40, 2, 4, 24, 32, False, True), (BF16, 40, 1, 1, 128, 128, True, True), (F32, 140, 1, 1, 128, 32, False, False),
    (BF16, 70, 1, 2, 40, 64, True, False), (F32, 44, 1, 2, 64, 64, True, True), (BF16, 130, 1, 3, 32, 32, False, True),
    (BF16, 70, 1, 2, 33, 64, False, True), (BF16, 70, 1, 2, 64, 64, True, True), (BF16, 150, 1, 1, 24, 64, False, True),
    (BF16, 70, 1, 1, 64, 128, False, False), (F32, 150, 1, 1, 64, 64, False, True),
    (F32, 150, 1, 1, 24, 64, True, True)])
def test_sequences_of_a_large_padded_batch(dt, B, Hk, H, dk, dv, reverse, s0):
    """Batches that are walked two tiles of columns at a time: each sequence as in a batch of its own."""
    print(f"\n[case] delta large {B} heads {Hk}/{H} {dk}x{dv} {dt}", flush=True)
    L = 130
    lens = [L - (37 * b) % (L + 9) for b in range(B)]
    c = Case(B, L, Hk, H, dk, dv, dt, reverse, lens, s0, seed=137)
    out = c.forward()
    gr = c.backward(out[2])
    for b in (0, 1, 3, B - 1):
        one = Case(1, L, Hk, H, dk, dv, dt, reverse, [lens[b]], s0)
        for n in ("q", "k", "v", "g", "beta", "do", "dl") + (("s0",) if s0 else ()):
            setattr(one, n, getattr(c, n)[b:b + 1].contiguous())
        o1 = one.forward()
        g1 = one.backward(o1[2])
        assert all(torch.equal(a[b:b + 1], x) for a, x in zip(out, o1))
        assert all(torch.equal(a[b:b + 1], x) for a, x in zip(gr, g1))
        if b == 1:
            one.check_forward(*o1)
            one.check_backward(g1)


def test_more_heads_than_a_row_of_the_grid():
    """2^18 and a few sequences: the last ones as in a batch of their own."""
    B, L, d = (1 << 18) + 21, 9, 8
    c = Case(64, L, 1, 1, d, d, BF16, seed=190)
    big = Case(1, 1, 1, 1, 1, 1, BF16)
    for n in ("q", "k", "v", "g", "beta", "s0", "do", "dl"):
        t = getattr(c, n)
        x = t[:1].expand(B, *t.shape[1:]).contiguous()
        x[-64:] = t
        setattr(big, n, x)
    out, want = big.forward(), c.forward()
    gr, wg = big.backward(out[2]), c.backward(want[2])
    for a, b in zip((*out, *gr), (*want, *wg)):
        assert torch.equal(a[-64:], b) and torch.equal(a[:5], b[:1].expand(5, *b.shape[1:]))
        assert torch.equal(a[1 << 17], b[0])


def test_refused_tensors():
    M = R()
    c = Case(2, 70, 1, 2, 16, 20, F32, seed=1)
    q, k, v, g, b = c.inputs()
    bad = [(q[:1], k, v, g, b), (q, k[..., :8], v, g, b), (q, k, v.bfloat16(), g, b), (q, k, v, g[:, :5], b),
           (q, k, v, g, b.cpu()), (q.half(), k, v, g, b), (q, k.transpose(0, 1).contiguous().transpose(0, 1), v, g, b),
           (q.repeat(1, 1, 3, 1), k.repeat(1, 1, 3, 1), v, g, b)]
    for args in bad:
        with pytest.raises(M.WbmmError):
            M.wbmm_delta_forward(*args)
        with pytest.raises(M.WbmmError):
            M.wbmm_delta_backward(*args, c.do)
    lens = torch.tensor([70, 3], dtype=torch.int32, device="cuda")
    states = c.forward()[2]
    for kw in (dict(s0=c.s0[:1]), dict(s0=c.s0.bfloat16()), dict(lens=lens.long()), dict(lens=lens[:1]), dict(o=v),
               dict(scale=float("inf")), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(M.WbmmError):
            M.wbmm_delta_forward(q, k, v, g, b, **kw)
    for kw in (dict(states=states[:, :, :1]), dict(states=states, s0=c.s0), dict(dv=c.do), dict(ds_last=c.dl[0]),
               dict(states=states, ds0=states[:, :, 0]), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(M.WbmmError):
            M.wbmm_delta_backward(q, k, v, g, b, c.do, **kw)


def test_offsets_past_32_bits():
    """Tensors of 4.3e9 bytes, and one sequence that is: its end equals a run from the states kept there."""
    for B, L in ((1030, 512), (1, 1030 * 512)):
        H, d = 32, 128
        mk = lambda *s: torch.empty(*s, dtype=BF16, device="cuda").normal_()  # noqa: E731
        q, k, v = mk(B, L, H, d), mk(B, L, H, d), mk(B, L, H, d)
        k *= d ** -0.5
        g, be = mk(B, L, H) + 2, mk(B, L, H)
        o, last, states = R().wbmm_delta_forward(q, k, v, g, be, s_last=True, states=B == 1)
        tail = 448
        cut = lambda t: t[-1:, L - tail:].contiguous()  # noqa: E731
        s0 = states[:, :, (L - tail) // 64].contiguous() if B == 1 else None
        if B > 1:
            part = lambda t: t[-1:].contiguous()  # noqa: E731
            o2, last2, _ = R().wbmm_delta_forward(part(q), part(k), part(v), part(g), part(be), s_last=True)
            assert torch.equal(o[-1:], o2) and torch.equal(last[-1:], last2)
        else:
            o2, last2, _ = R().wbmm_delta_forward(cut(q), cut(k), cut(v), cut(g), cut(be), s0=s0, s_last=True)
            assert torch.equal(cut(o), o2) and torch.equal(last, last2)
        del q, k, v, o, states, last
        torch.cuda.empty_cache()


def test_replayed_and_on_two_streams():
    cases = [Case(2, 150, 2, 4, 64, 48, BF16, seed=141), Case(3, 70, 1, 1, 32, 20, F32, lens=[70, 3, 64], seed=151)]

    def step(c):
        o, last, st = c.forward()
        return (o, last, st, *c.backward(st), *c.backward(None))

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = step(cases[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for n in range(3):
        new = Case(2, 150, 2, 4, 64, 48, BF16, seed=160 + n)
        for name in ("q", "k", "v", "g", "beta", "s0", "do", "dl"):
            getattr(c, name).copy_(getattr(new, name))
        want = step(c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_gradients_by_differences():
    """Central differences of the kernel's own forward in fp32. The loss is a sum of about 2 * 70 * 20 terms of
    size 1, good to 2^-24 of their sum of magnitudes (2^-24 * 256 of each by the bound above, at random: about
    16 of them in all); a difference over h = 2^-6 then errs by that over 2 h plus h^2 times a third derivative."""
    c = Case(1, 70, 1, 2, 16, 20, F32, seed=171)

    def loss():
        o, last, _ = c.forward(states=False)
        return float((o.double() * c.do.double()).sum() + (last.double() * c.dl.double()).sum())

    grads = c.backward(c.forward()[2])
    h = 2.0 ** -6
    for name, gr in zip(("q", "k", "v", "g", "beta", "s0"), grads):
        x = getattr(c, name)
        keep, d = x.clone(), torch.from_numpy(synth.normal_f32(tuple(x.shape), 1.0, 180)).cuda()
        d /= d.norm()
        x.copy_(keep + h * d)
        up = loss()
        x.copy_(keep - h * d)
        down = loss()
        x.copy_(keep)
        want = float((gr.double() * d.double()).sum())
        scale = float(gr.double().norm())
        assert abs((up - down) / (2 * h) - want) <= 1e-3 * scale + 1e-3, name


def wide(c):
    """The same case in fp32: bf16 values as they are."""
    w = Case(1, 1, 1, 1, 1, 1, F32)
    for n in ("q", "k", "v", "g", "beta", "do"):
        setattr(w, n, getattr(c, n).float())
    w.s0, w.dl, w.lens, w.hl, w.reverse, w.dk = c.s0, c.dl, c.lens, c.hl, c.reverse, c.dk
    return w


def overwritten(dk, dv, keys, times, old, beta):
    """`keys` keys written `times` times each over a state `old` times larger than what is written: what a
    query with the same key reads is a small difference of large products."""
    L = keys * times
    c = Case(1, L, 1, 1, dk, dv, BF16, gate=20.0, seed=201)
    c.k[:] = c.k[:, :keys].repeat(1, times, 1, 1)
    c.q, c.beta[:] = c.k.clone(), beta
    c.s0 *= old
    return c


BITS = SIZES + [(70, 130, 1, 1, 64, 128), (40, 130, 2, 4, 24, 32), (44, 70, 1, 2, 64, 64), (44, 70, 1, 1, 128, 128)]


def same_as_wide(name, c, states):
    w = wide(c)
    a, b = c.forward(states=states), w.forward(states=states)
    pairs = [("o", a[0], b[0]), ("s_last", a[1], b[1])]
    if states:
        pairs += [("states", a[2], b[2])]
        pairs += zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), c.backward(a[2]), w.backward(b[2]))
        pairs += zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), c.backward(None), w.backward(None))
    for n, x, y in pairs:
        y = y.to(x.dtype)
        assert torch.equal(x, y), (name, n, int((x != y).sum()), x.numel())


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("B,L,Hk,H,dk,dv", BITS)
def test_bf16_forward_is_the_fp32_one_rounded_once(B, L, Hk, H, dk, dv, reverse):
    """bf16 inputs are exact in fp32, and what is formed of them is held as in an fp32 call: its products and sums
    are the same ones, in the same order, so the results are the fp32 call's, rounded, bit for bit."""
    print(f"\n[case] delta bits {B}x{L} heads {Hk}/{H} {dk}x{dv} rev={reverse}", flush=True)
    same_as_wide("forward", Case(B, L, Hk, H, dk, dv, BF16, reverse, seed=211), False)


@pytest.mark.parametrize("dk,dv,keys,times,old,beta", [(64, 64, 8, 8, 1000.0, 6.0), (128, 48, 16, 4, 1.0, 8.0),
                                                       (33, 17, 5, 30, 1000.0, 6.0)])
def test_bf16_reads_of_overwritten_keys(dk, dv, keys, times, old, beta):
    c = overwritten(dk, dv, keys, times, old, beta)
    if old == 1.0:
        c.v.zero_()
    same_as_wide("overwritten", c, False)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("B,L,Hk,H,dk,dv", BITS)
def test_bf16_gradients_are_the_fp32_ones_rounded_once(B, L, Hk, H, dk, dv, reverse):
    print(f"\n[case] delta gradient bits {B}x{L} heads {Hk}/{H} {dk}x{dv} rev={reverse}", flush=True)
    same_as_wide("backward", Case(B, L, Hk, H, dk, dv, BF16, reverse, seed=221), True)


@pytest.mark.parametrize("dk,dv,keys,times,old,beta", [(64, 64, 8, 8, 1000.0, 6.0), (128, 48, 16, 4, 1.0, 8.0),
                                                       (33, 17, 5, 30, 1000.0, 6.0)])
def test_bf16_gradients_at_overwritten_keys(dk, dv, keys, times, old, beta):
    same_as_wide("overwritten", overwritten(dk, dv, keys, times, old, beta), True)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("L,dk,dv", [(70, 16, 20), (130, 64, 48), (64, 128, 32)])
def test_gradient_of_a_saturated_write_gate(L, dk, dv, dt):
    """beta of 10 to 20 and of -10 to -20: dbeta is (1 - b) times a dot product that errs by 256 half steps of its
    bound, dv M M_D, and 1 - b comes from an exponential, a sum and a quotient, 8 half steps of itself; so the
    smallest of them are as good as the largest."""
    c = Case(2, L, 1, 2, dk, dv, dt, seed=231)
    c.beta = (torch.from_numpy(synth.normal_f32((2, L, 2), 2.0, 232)).cuda().clamp(-5, 5) + 15).to(dt)
    c.beta[1] *= -1
    got = f64(c.backward(c.forward()[2])[4])
    x = [f64(t) for t in c.inputs()]
    M = K.delta_forward(*x, f64(c.s0), None, False, dk ** -0.5)[3]
    *w, MD, _ = K.delta_backward(*x, f64(c.s0), f64(c.do), f64(c.dl), None, False, dk ** -0.5)
    nb = 1 / (1 + np.exp(x[4]))
    want, h = w[4], half(dt)
    near("dbeta", got, want, 256 * U * dv * nb * (M * MD)[:, None] * (1 + h) + (8 * U + h) * np.abs(want))
    assert np.all(got[0] != 0) and np.abs(want[0]).max() > 100 * np.abs(want[0]).min() > 0


# With 3 as the gate at every size, and from nothing to everything at one.
GATES = [(s, 3.0) for s in SIZES] + [((2, 150, 1, 2, 32, 24), g) for g in (-100.0, -6.0, 0.0, 12.0, 100.0)]


def gate_bounds(x, s0, do, dl, lens, reverse, scale, want, h):
    """How far dg and dbeta of a head may be off in norm: the terms of their sums are dot products that err by 256 half
    steps of their factors' norms; the rest is a sum over 64 steps, the factors 1 - a and 1 - b (8 half
    steps) and a rounding to fp32, 16 half steps of the result in all, before its own rounding."""
    tg, tb, _ = K.delta_gate_bounds(*x, s0, do, dl, lens, reverse, scale)
    n = lambda t: np.sqrt((t * t).sum(1))  # noqa: E731
    return [256 * U * n(t) + (16 * U + h) * n(w) + 2.0 ** -126 * w.shape[1] ** 0.5 for t, w in zip((tg, tb), want)]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size,gate", GATES)
def test_gate_gradients_of_each_head(size, gate, dt, reverse):
    B, L, Hk, H, dk, dv = size
    print(f"\n[case] delta gates {size} {gate} {dt} rev={reverse}", flush=True)
    lens = [max(L - 7, 1)] * B if reverse else None
    c = Case(*size, dt, reverse, lens, gate=gate, seed=241)
    got = [f64(t) for t in c.backward(c.forward()[2])[3:5]]
    args = [f64(t) for t in c.inputs()], f64(c.s0), f64(c.do), f64(c.dl), lens, reverse, dk ** -0.5
    want = K.delta_backward(*args[0], *args[1:])[3:5]
    for name, x, w, tol in zip(("dg", "dbeta"), got, want, gate_bounds(*args, want, half(dt))):
        off = np.sqrt(((x - w) ** 2).sum(1))
        assert np.all(off <= tol), (name, off / tol)


@pytest.mark.parametrize("B,dv", [(64, 128), (70, 128), (90, 96), (180, 128)])
def test_large_batches_of_wide_keys(B, dv):
    """bf16 with 128 key entries, on either side of where a workgroup takes two tiles: each sequence as in a batch of its
    own, of which a tile is a workgroup's."""
    c = Case(B, 130, 1, 1, 128, dv, BF16, seed=251)
    out = c.forward()
    gr = c.backward(None)
    for b in (0, B // 2, B - 1):
        one = Case(1, 130, 1, 1, 128, dv, BF16)
        for n in ("q", "k", "v", "g", "beta", "s0", "do", "dl"):
            setattr(one, n, getattr(c, n)[b:b + 1].contiguous())
        assert all(torch.equal(a[b:b + 1], x) for a, x in zip((*out, *gr), (*one.forward(), *one.backward(None))))
