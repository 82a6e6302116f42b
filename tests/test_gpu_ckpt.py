"""8-bit activation checkpoints and the backward that reads them, on the GPU, against the fp64
oracles. Packing and unpacking are exact, so their comparisons are too."""
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


def values(n, seed):
    """fp32 values over many magnitudes, with the borders of the formats among them."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal(n) * np.exp(rng.standard_normal(n) * 4)).astype(np.float32)
    special = np.array([0, -0.0, 127, 127.5, 127.25, 448, 448.5, 464, 1e-45, 1.2e-38, 3e38, -3e38,
                        2.0 ** -126, 1.5 * 2.0 ** -9, 2.0 ** -10, 254, 63.5, 64], np.float32)
    at = rng.permutation(n)[: min(n, 5 * special.size)]
    x[at] = np.resize(special, at.size)
    if n > 40:
        x[n // 2: n // 2 + 20] = 0
    if n > 200:
        x[64:96] = 1e-42 * np.arange(32)     # a group of subnormal numbers
    return x


def check_pack(x, fmt, bf16, shape=None):
    if bf16:
        x = synth.round_to_bf16(x)
    t = dev(x).to(torch.bfloat16) if bf16 else dev(x)
    if shape:
        t = t.reshape(shape)
    codes, scales = R().wbmm_ckpt_pack(t, fmt=fmt)
    wc, ws = Q.pack(x.astype(np.float64), fmt)
    assert codes.shape == t.shape and np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy().reshape(-1), wc.reshape(-1))
    want = Q.unpack(wc, ws, fmt).reshape(-1)
    got = R().wbmm_ckpt_unpack(codes, scales, fmt=fmt)
    assert got.dtype == torch.float32 and got.shape == t.shape
    with np.errstate(over="ignore"):
        assert np.array_equal(got.cpu().numpy().reshape(-1), want.astype(np.float32), equal_nan=True)
    b = R().wbmm_ckpt_unpack(codes, scales, fmt=fmt, dtype=torch.bfloat16)
    assert torch.equal(b.nan_to_num(7.0), got.to(torch.bfloat16).nan_to_num(7.0))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 7, 31, 32, 33, 100, 511, 4096, 4097, 9001])
def test_pack_unpack_bit_exact(fmt, bf16, n):
    check_pack(values(n, n), fmt, bf16)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_pack_nonfinite_groups(fmt):
    x = values(200, 3)
    x[5], x[70], x[199] = np.inf, np.nan, -np.inf
    check_pack(x, fmt, False)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt,edge", [("int8", 127 / 64), ("e4m3", 31 / 16)])
def test_pack_largest_magnitudes(fmt, edge, bf16):
    """The largest values whose nearest code stands for a finite number, and those just above."""
    x = np.zeros(128, np.float32)
    top = np.float32(edge * 2.0 ** 127)
    step = np.float32(2.0 ** (120 if bf16 else 104))    # of the type, there
    below, above = (top, top + step) if fmt == "int8" else (top - step, top)
    x[3], x[40], x[70], x[100] = below, above, -below, -above
    check_pack(x, fmt, bf16)
    t = dev(x).to(torch.bfloat16 if bf16 else torch.float32)
    got = R().wbmm_ckpt_unpack(*R().wbmm_ckpt_pack(t, fmt=fmt), fmt=fmt).cpu().numpy()
    assert np.isfinite(got[[3, 70]]).all() and got[40] == np.inf and got[100] == -np.inf
    # half a step: of 127 even ones, or relative
    assert abs(got[3] / below - 1) <= (0.5 / 63.5 if fmt == "int8" else 2.0 ** -4)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_unpack_every_code_and_scale(fmt):
    codes = np.repeat(np.arange(256, dtype=np.uint8), 32).reshape(32 * 8, 32).T.copy().reshape(-1)
    codes = np.tile(np.arange(256, dtype=np.uint8), 256)       # every code under every scale
    scales = np.repeat(np.arange(256, dtype=np.uint8), 8)
    got = R().wbmm_ckpt_unpack(dev(codes), dev(scales), fmt=fmt).cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        want = Q.unpack(codes, scales, fmt).astype(np.float32)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("bf16,off", [(False, 1), (False, 3), (True, 1), (True, 4)])
def test_pack_at_odd_addresses(fmt, bf16, off):
    x = values(1000, 8)
    if bf16:
        x = synth.round_to_bf16(x)
    dt = torch.bfloat16 if bf16 else torch.float32
    base = torch.zeros(1100, dtype=dt, device="cuda")
    base[off:off + 1000] = dev(x).to(dt)
    codes = torch.full((1100,), 171, dtype=torch.uint8, device="cuda")
    scales = torch.full((64,), 171, dtype=torch.uint8, device="cuda")
    R().wbmm_ckpt_pack(base[off:off + 1000], fmt=fmt, codes=codes[off:off + 1000],
                       scales=scales[off:off + 32])
    wc, ws = Q.pack(x.astype(np.float64), fmt)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(c[off:off + 1000], wc) and np.array_equal(s[off:off + 32], ws)
    assert np.all(c[:off] == 171) and np.all(c[off + 1000:] == 171)
    assert np.all(s[:off] == 171) and np.all(s[off + 32:] == 171)
    out = torch.full((1100,), 9.0, dtype=dt, device="cuda")
    R().wbmm_ckpt_unpack(codes[off:off + 1000], scales[off:off + 32], fmt=fmt,
                         out=out[off:off + 1000])
    assert torch.all(out[:off] == 9) and torch.all(out[off + 1000:] == 9)
    want = torch.from_numpy(Q.unpack(wc, ws, fmt).astype(np.float32)).to(dt).cuda()
    assert torch.equal(out[off:off + 1000], want)


def bwd_inputs(B, C, H, W, w, mix, fmt, bf16, layout, seed):
    shape = (B, C, H, W) if layout == "NCHW" else (B, H, W, C)
    x = synth.normal_f32(shape, 1.0, seed)
    z = synth.normal_f32(shape, 0.02 * w, seed + 1)
    dy = synth.normal_f32(shape, 1.0, seed + 2)
    T = synth.normal_f32((C, 2 * w - 1, 2 * w - 1), 0.02, seed + 3)
    Wm = synth.normal_f32((C, 3, 3), 0.1, seed + 4) if mix else None
    if bf16:
        x, z, dy, T = (synth.round_to_bf16(v) for v in (x, z, dy, T))
    return x, z, dy, T, Wm


def nchw(a, layout):
    return a if layout == "NCHW" else np.ascontiguousarray(a.transpose(0, 3, 1, 2))


def check_bwd(B, C, H, W, w, mix, fmt, bf16, layout="NCHW", seed=0, **kw):
    print(f"\n[case] bwd_ckpt {B}x{C}x{H}x{W} w={w} mix={mix} {fmt} bf16={bf16} {layout}", flush=True)
    x, z, dy, T, Wm = bwd_inputs(B, C, H, W, w, mix, fmt, bf16, layout, seed)
    dt = torch.bfloat16 if bf16 else torch.float32
    pk = lambda a: R().wbmm_ckpt_pack(dev(a).to(dt), fmt=fmt)
    xc, zc = pk(x), pk(z) if mix else None
    un = lambda c: nchw(R().wbmm_ckpt_unpack(*c, fmt=fmt).cpu().numpy().astype(np.float64), layout)
    dx, dT, dW = R().wbmm_backward_ckpt(xc, dev(dy).to(dt), w, dev(T).to(dt),
                                        mix_w=dev(Wm) if mix else None, z_ckpt=zc, fmt=fmt,
                                        layout=layout, **kw)
    wdx, wdT, wdW = O.layer_backward(un(xc), nchw(dy, layout).astype(np.float64), w,
                                     T=T.astype(np.float64), Wmix=Wm, z=un(zc) if mix else None)
    if dx is not None:
        got = nchw(dx.float().cpu().numpy(), layout)
        if bf16:   # fp32 arithmetic, then one rounding of half a bf16 step
            err = np.abs(got - wdx)
            assert np.all(err <= 2.0 ** -8 * np.abs(wdx) + 1e-5), err.max()
        else:
            assert_f32(got, wdx, "dx")
    if dT is not None:
        assert_f32(dT.cpu().numpy(), wdT, "dT")
    if dW is not None:
        assert_f32(dW.cpu().numpy(), wdW, "dWmix")
    return dx, dT, dW


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,C,H,W,w", [
    (5, 3, 28, 28, 14), (3, 2, 56, 56, 14), (18, 3, 14, 14, 14),   # whole-image kernels, part units
    (1, 1, 28, 28, 14), (2, 3, 30, 45, 7), (3, 5, 9, 9, 3), (2, 3, 5, 40, 8), (2, 2, 20, 20, 16),
    (2, 2, 30, 20, 20), (1, 2, 4, 5, 14),
])
def test_backward_ckpt(fmt, bf16, mix, B, C, H, W, w):
    check_bwd(B, C, H, W, w, mix, fmt, bf16, seed=B + w)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,C,H", [(64, 2, 28), (33, 3, 56), (97, 2, 14), (8, 1, 28), (9, 1, 28),
                                   (2, 1, 56), (3, 1, 56), (32, 1, 14), (33, 1, 14)])
def test_backward_ckpt_whole_images(B, C, H, mix, bf16):
    """Many units of the fused kernel, and units with one image or all but one missing."""
    check_bwd(B, C, H, H, 14, mix, "int8", bf16, seed=H + B)


@pytest.mark.parametrize("bf16", [False, True])
def test_backward_ckpt_misaligned_buffers(bf16):
    """Buffers that the fused kernel's wide accesses cannot take go through the general kernels."""
    B, C, H, w = 9, 3, 28, 14
    x, z, dy, T, Wm = bwd_inputs(B, C, H, H, w, True, "int8", bf16, "NCHW", 3)
    dt = torch.bfloat16 if bf16 else torch.float32
    (xc, xs), (zc, zs) = (R().wbmm_ckpt_pack(dev(a).to(dt)) for a in (x, z))
    kw = dict(mix_w=dev(Wm), w=w, T=dev(T).to(dt))
    want = R().wbmm_backward_ckpt((xc, xs), dev(dy).to(dt), z_ckpt=(zc, zs), **kw)

    def moved(t, by=1):
        buf = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        out = buf[by:by + t.numel()].view(t.shape)
        out.copy_(t)
        return out

    dyd = dev(dy).to(dt)
    for args in (dict(x_ckpt=(moved(xc), xs), dy=dyd, z_ckpt=(zc, zs)),
                 dict(x_ckpt=(xc, moved(xs)), dy=dyd, z_ckpt=(moved(zc, 3), zs)),
                 dict(x_ckpt=(xc, xs), dy=moved(dyd), z_ckpt=(zc, zs)),
                 dict(x_ckpt=(xc, xs), dy=dyd, z_ckpt=(zc, zs), dx=moved(dyd))):
        got = R().wbmm_backward_ckpt(**args, **kw)
        assert_f32(got[1].cpu().numpy(), want[1].double().cpu().numpy(), "dT")
        assert_f32(got[2].cpu().numpy(), want[2].double().cpu().numpy(), "dW")
        a, b = got[0].double(), want[0].double()
        half = 2.0 ** -8 if bf16 else 2.0 ** -22    # each side rounds once
        assert torch.all((a - b).abs() <= 2 * half * b.abs() + 1e-5)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("w", range(1, 18))
def test_backward_ckpt_every_window(w, bf16):
    """A ragged map for every window side, with windows of several images in a unit of 32."""
    check_bwd(3, 2, 2 * w + max(1, w // 2), 3 * w - w // 3, w, True, "e4m3", bf16, seed=w)
    check_bwd(1, 1, w, w, w, False, "int8", bf16, seed=w)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,C,H,W,w", [(40, 70, 17, 15, 3), (3, 1, 200, 210, 2), (64, 3, 30, 45, 7),
                                       (2, 5, 140, 100, 14), (70, 66, 12, 12, 4)])
def test_backward_ckpt_many_units(B, C, H, W, w, bf16):
    """Workgroups that take several units, and channels with many workgroups."""
    check_bwd(B, C, H, W, w, True, "int8", bf16, seed=w)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,C,H,W,w,layout", [(33, 60, 22, 30, 16, "NCHW"), (66, 90, 11, 19, 11, "NHWC")])
def test_backward_ckpt_many_units_of_large_windows(B, C, H, W, w, layout, bf16):
    """One workgroup per CU and more units than CUs: some take several."""
    check_bwd(B, C, H, W, w, True, "int8", bf16, layout=layout, seed=w)


@pytest.mark.parametrize("C,H,W,w", [(2, 4030, 4031, 16), (1, 5704, 5709, 5)])
def test_backward_ckpt_largest_images(C, H, W, w):
    """Images on either side of the size up to which a unit's offsets take 32 bits (33 images of
    2^32 bytes): the gradients of the decoded maps.

    Both sides round each of a sum's n terms by a few 2^-24 of it, in chains of fp32 and then fp64: the
    error's norm stays below 2^-20 of the root of the terms' squares, which is what the sums of these
    random terms measure themselves, and 2e-6 leaves twice that."""
    assert (4 * 33 * C * H * W < 2 ** 32) == (C == 2)
    x, z, dy, T, Wm = bwd_inputs(1, C, H, W, w, True, "int8", False, "NCHW", 5)
    xc, zc = (R().wbmm_ckpt_pack(dev(a)) for a in (x, z))
    xu, zu = (R().wbmm_ckpt_unpack(*c) for c in (xc, zc))
    got = R().wbmm_backward_ckpt(xc, dev(dy), w, dev(T), mix_w=dev(Wm), z_ckpt=zc)
    want = R().wbmm_backward(xu, dev(dy), w, T=dev(T), mix_w=dev(Wm), z_saved=zu)
    for a, b, name in zip(got, want, ("dx", "dT", "dW")):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= 2e-6 * b.norm(), name


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,C,H,W,w", [(2, 12, 17, 19, 7), (3, 5, 28, 28, 14), (2, 3, 5, 6, 8)])
def test_backward_ckpt_nhwc(B, C, H, W, w, bf16, mix):
    check_bwd(B, C, H, W, w, mix, "int8", bf16, layout="NHWC")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("H,W,w", [(30, 45, 7), (13, 9, 5), (28, 28, 14), (20, 33, 16)])
def test_backward_ckpt_writes_only_its_outputs(H, W, w, bf16):
    B, C, G = 3, 2, 61
    x, z, dy, T, Wm = bwd_inputs(B, C, H, W, w, True, "int8", bf16, "NCHW", 1)
    dt = torch.bfloat16 if bf16 else torch.float32
    xc, zc = (R().wbmm_ckpt_pack(dev(a).to(dt)) for a in (x, z))
    bufs = []

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * G,), 33.0, dtype=dtype, device="cuda")
        bufs.append(buf)
        out = buf[G:G + n].view(shape)
        out.fill_(float("nan"))
        return out

    L = 2 * w - 1
    outs = (guarded(dy.shape, dt), guarded((C, L, L), torch.float32), guarded((C, 3, 3), torch.float32))
    need = R().wbmm_backward_ckpt_workspace_bytes(B, C, H, W, w, dtype=dt, has_mix=True)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    R().wbmm_backward_ckpt(xc, dev(dy).to(dt), w, dev(T).to(dt), mix_w=dev(Wm), z_ckpt=zc, dx=outs[0],
                           dT=outs[1], dmix_w=outs[2], workspace=ws[:need])
    for t in outs:
        assert torch.isfinite(t.float()).all()
    for b in bufs:
        assert torch.all(b[:G] == 33) and torch.all(b[-G:] == 33)
    assert torch.all(ws[need:] == 77)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,H,w", [(5, 28, 14), (2, 13, 5)])
def test_backward_ckpt_partial_outputs(bf16, B, H, w):
    """Each output alone is what the whole call gives."""
    whole = check_bwd(B, 3, H, H, w, True, "int8", bf16, seed=4)
    for k in range(3):
        flags = dict(dx=k == 0, dT=k == 1, dmix_w=k == 2)
        part = check_bwd(B, 3, H, H, w, True, "int8", bf16, seed=4, **flags)
        for j in range(3):
            assert (part[j] is None) == (j != k)
        assert torch.equal(part[k], whole[k])


@pytest.mark.parametrize("B,C,H,W,w", [(76800, 1, 28, 28, 7), (12800, 1100, 7, 7, 7), (3000, 1, 160, 160, 16)])
def test_backward_ckpt_mix_gradient_of_many_units(B, C, H, W, w):
    """dWmix where a workgroup takes hundreds of units (one channel, or more than a thousand), all terms
    equal, so that every rounding of a sum falls the same way. A thread's fp32 sum holds 128 terms at
    most, then come 4 sums of lanes, fp64 and dWmix's own rounding: 133 half steps."""
    dy = torch.full((B, C, H, W), 1.9153239727020264, device="cuda")
    x = R().wbmm_ckpt_pack(torch.zeros_like(dy))
    z = R().wbmm_ckpt_pack(torch.full_like(dy, 0.75))
    T = torch.zeros(C, 2 * w - 1, 2 * w - 1, device="cuda")
    mix = torch.zeros(C, 3, 3, device="cuda")
    dW = R().wbmm_backward_ckpt(x, dy, w, T, mix_w=mix, z_ckpt=z, dx=False, dT=False)[2]
    rows = np.array([H - 1, H, H - 1], np.float64)[:, None] * np.array([W - 1, W, W - 1], np.float64)
    want = B * rows * 0.75 * float(dy.view(-1)[0])
    worst = np.max(np.abs(dW.double().cpu().numpy() / want - 1)) * 2.0 ** 24
    print(f"    dW: worst {worst:.1f} half steps", flush=True)
    assert worst <= 133


@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("B,C,H,W,w", [(5, 3, 28, 28, 14), (2, 3, 30, 45, 7), (2, 2, 30, 40, 20)])
def test_backward_ckpt_bf16_dx_error(B, C, H, W, w, mix):
    """dx of bf16 maps, element by element, against what may be lost, U = 2^-24: half a step of the
    result; with the mix 2^-17 of each G, and 9 U of the adjoint's terms for its 9 sums; U for each
    of the up to 2 w^2 products (a part of G each) that a sum takes, and one more for the two parts."""
    x, z, dy, T, Wm = bwd_inputs(B, C, H, W, w, mix, "int8", True, "NCHW", 21)
    pk = lambda a: R().wbmm_ckpt_pack(dev(a).to(torch.bfloat16))
    dx = R().wbmm_backward_ckpt(pk(x), dev(dy).to(torch.bfloat16), w, dev(T).to(torch.bfloat16),
                                mix_w=dev(Wm) if mix else None, z_ckpt=pk(z) if mix else None)[0]
    f = lambda a: None if a is None else a.astype(np.float64)
    b = lambda a: None if a is None else np.abs(f(a))
    zz = f(z) if mix else None
    want = O.layer_backward(f(x), f(dy), w, T=f(T), Wmix=f(Wm), z=zz)[0]
    terms = O.layer_backward(f(x), b(dy), w, T=b(T), Wmix=b(Wm), z=zz)[0]
    U = 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(want) + terms * ((2.0 ** -17 + 9 * U if mix else 0) + (2 * w * w + 1) * U)
    err = np.abs(dx.double().cpu().numpy() - want)
    print(f"    dx: worst error/bound {np.max(err / tol):.3f}", flush=True)
    assert np.all(err <= tol * (1 + 2.0 ** -8))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_backward_ckpt_is_the_backward_of_the_decoded_maps(fmt):
    """fp32: the same gradients as wbmm_backward on the unpacked maps, to rounding."""
    x, z, dy, T, Wm = bwd_inputs(9, 4, 28, 28, 14, True, fmt, False, "NCHW", 11)
    xc, zc = (R().wbmm_ckpt_pack(dev(a), fmt=fmt) for a in (x, z))
    un = lambda c: R().wbmm_ckpt_unpack(*c, fmt=fmt)
    got = R().wbmm_backward_ckpt(xc, dev(dy), 14, dev(T), mix_w=dev(Wm), z_ckpt=zc, fmt=fmt)
    want = R().wbmm_backward(un(xc), dev(dy), 14, T=dev(T), mix_w=dev(Wm), z_saved=un(zc))
    for a, b, name in zip(got, want, ("dx", "dT", "dW")):
        assert_f32(a.cpu().numpy(), b.double().cpu().numpy(), name)


def test_backward_ckpt_nan_group_reaches_its_channel_only():
    x, z, dy, T, Wm = bwd_inputs(2, 3, 28, 28, 14, False, "int8", False, "NCHW", 1)
    x[0, 1, 3, 3] = np.inf
    xc = R().wbmm_ckpt_pack(dev(x))
    dx, dT, _ = R().wbmm_backward_ckpt(xc, dev(dy), 14, dev(T))
    assert torch.isfinite(dx).all() and torch.isfinite(dT[[0, 2]]).all()
    assert torch.isnan(dT[1]).any()


def test_backward_ckpt_determinism_stream_and_graph():
    x, z, dy, T, Wm = bwd_inputs(17, 6, 28, 28, 14, True, "int8", False, "NCHW", 2)
    xc, zc = (R().wbmm_ckpt_pack(dev(a)) for a in (x, z))
    args = (xc, dev(dy), 14, dev(T))
    kw = dict(mix_w=dev(Wm), z_ckpt=zc)
    want = R().wbmm_backward_ckpt(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = R().wbmm_backward_ckpt(*args, stream=side, **kw)
    side.synchronize()
    for a, b in zip(on_side, want):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = R().wbmm_backward_ckpt(*args, **kw)
    for k in range(3):
        for t in out:
            t.fill_(float(k))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_binding_refusals():
    M = R()
    x = torch.zeros(2, 3, 28, 28, device="cuda")
    codes, scales = M.wbmm_ckpt_pack(x)
    T = torch.zeros(3, 27, 27, device="cuda")
    bad = [
        lambda: M.wbmm_ckpt_pack(x.cpu()), lambda: M.wbmm_ckpt_pack(x, fmt="fp4"),
        lambda: M.wbmm_ckpt_pack(x.half()), lambda: M.wbmm_ckpt_pack(x[..., ::2]),
        lambda: M.wbmm_ckpt_pack(x[:0]), lambda: M.wbmm_ckpt_pack(x, codes=codes[:1]),
        lambda: M.wbmm_ckpt_unpack(codes, scales[:-1]),
        lambda: M.wbmm_ckpt_unpack(codes.float(), scales),
        lambda: M.wbmm_backward_ckpt((codes, scales), x.bfloat16(), 14, T),
        lambda: M.wbmm_backward_ckpt((codes, scales), x, 7, T),
        lambda: M.wbmm_backward_ckpt((codes, scales), x, 14, T, z_ckpt=(codes, scales)),
        lambda: M.wbmm_backward_ckpt((codes[:1], scales), x, 14, T),
        lambda: M.wbmm_backward_ckpt((codes, scales), x, 14, T, dx=x),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(M.WbmmError):
            f()
            pytest.fail(f"call {k} was accepted")
