"""A training step of a windowed layer followed by the recurrence over its map, keeping 8 bits of x, z
and u between forward and backward: the calls in the order a program makes them, each result against
the fp64 oracles on what the call was given, eagerly and replayed from a graph."""
import numpy as np
import pytest

from oracle import ops_oracle as Q
from oracle import wbmm_oracle as O
from receptive_field_spatial_amd import synth
from tests.parity_util import assert_f32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def R():
    import receptive_field_spatial_amd as mod
    mod.load_library()
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Step:
    """One layer and one recurrence on (B, C, H, W) or (B, H, W, C) maps."""

    def __init__(self, B, C, H, W, w, layout, fmt, dtype, reverse, seed):
        shape = (B, C, H, W) if layout == "NCHW" else (B, H, W, C)
        mk = lambda s, sig, k: dev(synth.normal_f32(s, sig, seed + k)).to(dtype)
        self.w, self.layout, self.fmt, self.reverse, self.dtype = w, layout, fmt, reverse, dtype
        self.x, self.dh = mk(shape, 1.0, 0), mk(shape, 1.0, 1)
        self.g = mk(shape, 1.0, 2) + 2
        self.T = mk((C, 2 * w - 1, 2 * w - 1), 0.05, 3)
        self.mix = dev(synth.normal_f32((C, 3, 3), 0.3, seed + 4))
        # raster order: (B, C, H W) along the last axis, or (B, H W, C) along the middle one
        self.flat = (B, C, H * W) if layout == "NCHW" else (B, H * W, C)
        self.dim = 2 if layout == "NCHW" else 1

    def run(self):
        M = R()
        z = torch.empty_like(self.x)
        y = M.wbmm_forward(self.x, self.w, T=self.T, mix_w=self.mix, z_save=z, layout=self.layout)
        seq = lambda t: t.view(self.flat)
        h, last, st = M.wbmm_scan_forward(seq(self.g), seq(y), self.dim, reverse=self.reverse,
                                          h_last=True, states=True)
        pk = lambda t: M.wbmm_ckpt_pack(t, fmt=self.fmt)
        xc, zc, uc = pk(self.x), pk(z), pk(seq(y))
        # from here on x, z, y are gone: the checkpoints and the gate are what a step keeps
        dg, du, d0 = M.wbmm_scan_backward(seq(self.g), None, seq(self.dh), self.dim, u_ckpt=uc,
                                          fmt=self.fmt, reverse=self.reverse)
        dx, dT, dW = M.wbmm_backward_ckpt(xc, du.view(self.x.shape), self.w, self.T, mix_w=self.mix,
                                          z_ckpt=zc, fmt=self.fmt, layout=self.layout)
        return dict(y=y, h=h, last=last, st=st, dg=dg, du=du, d0=d0, dx=dx, dT=dT, dW=dW, xc=xc[0],
                    xs=xc[1], zc=zc[0], zs=zc[1], uc=uc[0], us=uc[1])

    def check(self, r):
        bf16 = self.dtype == torch.bfloat16
        half = 2.0 ** -8 if bf16 else 2.0 ** -24
        sh = self.flat if self.dim == 1 else (self.flat[0] * self.flat[1], self.flat[2], 1)
        seq = lambda t: f64(t).reshape(sh)

        def near(got, want, bound, h):
            assert np.all(np.abs(got - want) <= bound * (1 + h) + h * np.abs(want) + 1e-36)

        wh, wl, wst, bh, bl, bst = Q.scan_forward(seq(self.g), seq(r["y"]), None, None, self.reverse, bf16)
        near(seq(r["h"]), wh, bh, half)
        near(f64(r["last"]).reshape(wl.shape), wl, bl, 2.0 ** -24)
        near(f64(r["st"]).reshape(wst.shape), wst, bst, 2.0 ** -24)
        val = lambda c, s: Q.unpack(c.cpu().numpy(), s.cpu().numpy(), self.fmt)
        u = val(r["uc"], r["us"]).reshape(sh)
        wdg, wdu, wd0, bg, bu, b0 = Q.scan_backward(seq(self.g), u, None, seq(self.dh), None, None,
                                                    self.reverse, bf16)
        near(seq(r["dg"]), wdg, bg, half)
        near(seq(r["du"]), wdu, bu, half)
        near(f64(r["d0"]).reshape(wd0.shape), wd0, b0, 2.0 ** -24)
        nchw = lambda a: a if self.layout == "NCHW" else np.ascontiguousarray(a.transpose(0, 3, 1, 2))
        wdx, wdT, wdW = O.layer_backward(
            nchw(val(r["xc"], r["xs"])), nchw(f64(r["du"]).reshape(self.x.shape)), self.w, T=f64(self.T),
            Wmix=f64(self.mix), z=nchw(val(r["zc"], r["zs"])))
        dx = nchw(f64(r["dx"]))
        if bf16:
            assert np.all(np.abs(dx - wdx) <= half * np.abs(wdx) + 1e-5)
        else:
            assert_f32(dx, wdx, "dx")
        assert_f32(r["dT"].cpu().numpy(), wdT, "dT")
        assert_f32(r["dW"].cpu().numpy(), wdW, "dWmix")


CASES = [
    (4, 3, 28, 28, 14, "NCHW", "int8", torch.float32, False),
    (3, 4, 28, 28, 14, "NCHW", "e4m3", torch.bfloat16, True),
    (2, 6, 17, 11, 5, "NHWC", "int8", torch.float32, True),
    (2, 5, 9, 16, 7, "NHWC", "e4m3", torch.bfloat16, False),
    (1, 3, 30, 45, 7, "NCHW", "e4m3", torch.float32, False),
]


@pytest.mark.parametrize("B,C,H,W,w,layout,fmt,dtype,reverse", CASES)
def test_training_step(B, C, H, W, w, layout, fmt, dtype, reverse):
    print(f"\n[case] step {B}x{C}x{H}x{W} w={w} {layout} {fmt} {dtype} rev={reverse}", flush=True)
    s = Step(B, C, H, W, w, layout, fmt, dtype, reverse, seed=5)
    s.check(s.run())


@pytest.mark.parametrize("B,C,H,W,w,layout,fmt,dtype,reverse", CASES[:3])
def test_training_step_replayed(B, C, H, W, w, layout, fmt, dtype, reverse):
    """The whole step captured once and replayed on new inputs, with eager steps in between."""
    s = Step(B, C, H, W, w, layout, fmt, dtype, reverse, seed=6)
    other = Step(B, C, H, W, w, layout, fmt, dtype, reverse, seed=7)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run()
    for k in range(3):
        src = other if k % 2 == 0 else Step(B, C, H, W, w, layout, fmt, dtype, reverse, seed=8)
        for name in ("x", "dh", "g", "T", "mix"):
            getattr(s, name).copy_(getattr(src, name))
        want = src.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in want.items():
            assert torch.equal(out[name], t), name


def test_two_streams_at_once():
    """The same step on two streams, each call with its own workspace."""
    steps = [Step(*CASES[k][:8], CASES[k][8], seed=9 + k) for k in (0, 2)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = steps[k].run()
    torch.cuda.synchronize()
    for k in range(2):
        for name, t in want[k].items():
            assert torch.equal(got[k][name], t), name
