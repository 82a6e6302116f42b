"""A training step of a block: norm (kept in 8 bits for the layer's backward), windowed layer, norm joined
with the residual, delta rule over the map in raster order, the gradients of all of them and AdamW over the
block's parameters, as a program makes the calls; against the fp64 oracles chained in the same way, eagerly,
replayed from a graph and on two streams at once.

Tolerance. Each of the nine results of a pass is good to about 256 half steps of fp32 relative to its norm
(bf16 maps: and half a step of bf16 per map stored), and errors pass through norms and contractions that
enlarge them by less than 2 each: 9 * 2 * 256 * 2^-24 < 2^-11 at the end of the chain, bf16 2^-11 +
4 * 2 * 2^-8 = 2^-5."""
import numpy as np
import pytest

from oracle import block_oracle as K
from oracle import wbmm_oracle as O
from receptive_field_spatial_amd import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32, BF16 = torch.float32, torch.bfloat16


def R():
    import receptive_field_spatial_amd as mod
    mod.load_library()
    return mod


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Block:
    def __init__(self, B, H, W, heads, d, w, dtype, fmt, small, seed):
        C = heads * d
        mk = lambda s, sig, k: torch.from_numpy(synth.normal_f32(s, sig, seed + k)).cuda()  # noqa: E731
        unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(dtype)  # noqa: E731
        self.w, self.fmt, self.dtype, self.heads, self.d = w, fmt, dtype, heads, d
        self.shape, L = (B, H, W, C), H * W
        self.x, self.r = mk(self.shape, 1.0, 0).to(dtype), mk(self.shape, 1.0, 1).to(dtype)
        self.q, self.k = unit(mk((B, L, 1, 24), 1.0, 2)), unit(mk((B, L, 1, 24), 1.0, 3))
        self.g, self.beta = (mk((B, L, heads), 1.0, 4) + 2).to(dtype), mk((B, L, heads), 1.0, 5).to(dtype)
        self.do = mk((B, L, heads, d), 1.0, 6).to(dtype)
        n = 2 * w - 1
        self.params = [mk((C, n, n), 0.05, 7), mk((C, 3, 3), 0.3, 8), 1 + mk((C,), 0.1, 9), 1 + mk((C,), 0.1, 10)]
        self.grads = [torch.zeros_like(p) for p in self.params]

        def state(p):
            if not small:
                return torch.zeros_like(p)
            return (torch.zeros(p.shape, dtype=torch.uint8, device="cuda"),
                    torch.zeros(-(-p.numel() // 32), dtype=torch.uint8, device="cuda"))

        self.m, self.v = [state(p) for p in self.params], [state(p) for p in self.params]
        self.copies = [torch.zeros(p.shape, dtype=BF16, device="cuda") for p in self.params]
        self.plan = R().wbmm_adamw_plan(self.params, self.grads, self.m, self.v, copies=self.copies,
                                        weight_decay=[0.0, 0.01, 0.0, 0.0])
        self.step_count = torch.zeros(1, dtype=torch.int32, device="cuda")

    def gradients(self):
        M = R()
        T, mix, w1, w2 = self.params
        dT, dmix, dw1, dw2 = self.grads
        lay = T.to(self.dtype)       # the layer takes its table in the maps' type
        y1, s1, ck = M.wbmm_rmsnorm_forward(self.x, 3, residual=self.r, weight=w1, fmt=self.fmt)
        z = torch.empty_like(self.x)
        a = M.wbmm_forward(y1, self.w, T=lay, mix_w=mix, z_save=z, layout="NHWC")
        y2, s2, _ = M.wbmm_rmsnorm_forward(a, 3, residual=s1, weight=w2)
        seq = lambda t: t.view(self.do.shape)  # noqa: E731
        o, last, st = M.wbmm_delta_forward(self.q, self.k, seq(y2), self.g, self.beta, s_last=True, states=True)
        zc = M.wbmm_ckpt_pack(z, fmt=self.fmt)
        dq, dk, dy2, dg, dbeta, _ = M.wbmm_delta_backward(self.q, self.k, seq(y2), self.g, self.beta, self.do, states=st,
                                                          ds_last=last, ds0=False)
        ds2, _ = M.wbmm_rmsnorm_backward(s2, dy2.view(self.shape), 3, weight=w2, dweight=dw2)
        dy1, gT, gmix = M.wbmm_backward_ckpt(ck, ds2, self.w, lay, mix_w=mix, z_ckpt=zc, fmt=self.fmt, layout="NHWC")
        dx, _ = M.wbmm_rmsnorm_backward(s1, dy1, 3, weight=w1, ds=ds2, dweight=dw1)
        dT.copy_(gT)
        dmix.copy_(gmix)
        return dict(y1=y1, s1=s1, a=a, y2=y2, o=o, last=last, dq=dq, dk=dk, dg=dg, dbeta=dbeta, dx=dx, dT=dT, dmix=dmix,
                    dw1=dw1, dw2=dw2), ck, zc

    def step(self):
        out, ck, zc = self.gradients()
        self.step_count.add_(1)
        R().wbmm_adamw_step(self.plan, lr=1e-3, step=self.step_count, seed=9)
        return [*out.values(), *self.params, *self.copies,
                *[t for s in self.m + self.v for t in (s if isinstance(s, tuple) else (s,))]]

    def oracle(self, ck, zc):
        """The same from the inputs, in fp64; the layer's backward reads the 8-bit values, as it does there."""
        C = self.shape[3]
        T, mix, w1, w2 = [f64(p) for p in self.params]
        T = f64(self.params[0].to(self.dtype))
        rows = lambda t: t.reshape(-1, C, 1)  # noqa: E731
        maps = lambda t: t.reshape(self.shape)  # noqa: E731
        nchw = lambda t: maps(t).transpose(0, 3, 1, 2)  # noqa: E731
        nhwc = lambda t: np.ascontiguousarray(t.transpose(0, 2, 3, 1))  # noqa: E731
        back = lambda c: f64(R().wbmm_ckpt_unpack(*c, fmt=self.fmt))  # noqa: E731
        s1, y1 = K.norm_forward(rows(f64(self.x)), rows(f64(self.r)), w1, 1e-6)
        a = nhwc(O.layer_forward(nchw(y1), self.w, T=T, Wmix=mix)[0])
        s2, y2 = K.norm_forward(rows(a), s1, w2, 1e-6)
        x = [f64(t) for t in (self.q, self.k)] + [y2.reshape(self.do.shape)] + [f64(t) for t in (self.g, self.beta)]
        scale = 24 ** -0.5
        o, last, _, _ = K.delta_forward(*x, None, None, False, scale)
        dq, dk, dy2, dg, dbeta, _, _, _ = K.delta_backward(*x, None, f64(self.do), last, None, False, scale)
        ds2, dw2, _, _ = K.norm_backward(s2, rows(dy2), None, w2, 1e-6)
        dy1, dT, dmix = O.layer_backward(nchw(back(ck)), nchw(ds2), self.w, T=T, Wmix=mix, z=nchw(back(zc)))[:3]
        dx, dw1, _, _ = K.norm_backward(s1, rows(nhwc(dy1)), ds2, w1, 1e-6)
        return dict(y1=maps(y1), s1=maps(s1), a=a, y2=maps(y2), o=o, last=last, dq=dq, dk=dk, dg=dg, dbeta=dbeta,
                    dx=maps(dx), dT=dT, dmix=dmix, dw1=dw1, dw2=dw2)


CASES = [(2, 14, 14, 2, 16, 7, F32, "int8", False), (1, 15, 9, 3, 20, 5, F32, "e4m3", True),
         (2, 14, 21, 2, 32, 7, BF16, "e4m3", True)]


@pytest.mark.parametrize("B,H,W,heads,d,w,dtype,fmt,small", CASES)
def test_step_against_the_oracles(B, H, W, heads, d, w, dtype, fmt, small):
    b = Block(B, H, W, heads, d, w, dtype, fmt, small, 1)
    got, ck, zc = b.gradients()
    want = b.oracle(ck, zc)
    tol = 2.0 ** -11 if dtype == F32 else 2.0 ** -5
    for name, t in want.items():
        err = np.linalg.norm(f64(got[name]) - t) / np.linalg.norm(t)
        assert err <= tol, (name, err)


@pytest.mark.parametrize("B,H,W,heads,d,w,dtype,fmt,small", CASES)
def test_step_replayed(B, H, W, heads, d, w, dtype, fmt, small):
    a, b = (Block(B, H, W, heads, d, w, dtype, fmt, small, 1) for _ in range(2))
    a.step(), b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a.step()
    for k in range(3):
        for t in (a, b):
            t.x.copy_(torch.from_numpy(synth.normal_f32(t.shape, 1.0, 100 + k)))
        want = b.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert int(a.step_count) == 4


def test_two_blocks_on_two_streams():
    alone = [Block(*c, 20 + i) for i, c in enumerate(CASES[1:])]
    want = []
    for b in alone:
        for _ in range(3):
            out = b.step()
        want.append([t.clone() for t in out])
    both = [Block(*c, 20 + i) for i, c in enumerate(CASES[1:])]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = both[i].step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a, b in zip(want, got) for x, y in zip(a, b))


def test_steps_go_downhill_along_the_gradient():
    """The loss of the block, <o, do>, by differences along a random direction of the parameters: fp32, the
    8-bit values apart, which the layer's own weight gradients see (int8: 2^-7 of each value at most, a random
    sum of many: 2^-5 of the whole is more than enough); h^2 and rounding errors are below 2^-8."""
    b = Block(2, 14, 14, 2, 16, 7, F32, "int8", False, 41)

    def loss():
        M, (T, mix, w1, w2) = R(), b.params
        y1, s1, _ = M.wbmm_rmsnorm_forward(b.x, 3, residual=b.r, weight=w1)
        y2, _, _ = M.wbmm_rmsnorm_forward(M.wbmm_forward(y1, b.w, T=T, mix_w=mix, layout="NHWC"), 3, residual=s1, weight=w2)
        o, last, _ = M.wbmm_delta_forward(b.q, b.k, y2.view(b.do.shape), b.g, b.beta, s_last=True)
        return float((o.double() * b.do.double()).sum() + last.double().square().sum() / 2)

    b.gradients()
    h = 2.0 ** -7
    for i, (p, g) in enumerate(zip(b.params, b.grads)):
        d = torch.from_numpy(synth.normal_f32(tuple(p.shape), 1.0, 60 + i)).cuda()
        d = d / d.norm() + g / g.norm()      # half of it along the gradient: a slope that differences see
        keep = p.clone()
        p.copy_(keep + h * d)
        up = loss()
        p.copy_(keep - h * d)
        down = loss()
        p.copy_(keep)
        want = float((g.double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) <= (2.0 ** -5 + 2.0 ** -8) * float(g.double().norm()), i
