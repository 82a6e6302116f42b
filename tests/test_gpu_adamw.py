"""AdamW over many tensors. The step is defined operation by operation in fp32, so that it equals the
oracle bit for bit, 8-bit states included; the fp64 step stands beside it."""
import numpy as np
import pytest

from oracle import block_oracle as K
from receptive_field_spatial_amd import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
KW = dict(lr=1e-2, b1=0.9, b2=0.99, eps=1e-8)


def R():
    import receptive_field_spatial_amd as mod
    mod.load_library()
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def zeros8(n):
    return torch.zeros(n, dtype=U8, device="cuda"), torch.zeros(-(-n // 32), dtype=U8, device="cuda")


class Model:
    """Tensors of different sizes, gradient types, states and copies; `shift` puts every buffer that many
    elements past an aligned address."""

    def __init__(self, spec, seed, shift=0):
        self.p, self.g, self.m, self.v, self.copy, self.wd = [], [], [], [], [], []
        for k, (n, gdt, small, copy, wd) in enumerate(spec):
            put = lambda t: torch.cat([torch.zeros(shift, dtype=t.dtype, device="cuda"), t])[shift:]  # noqa: E731
            self.p.append(put(dev(synth.normal_f32((n,), 0.5, seed + 7 * k))))
            self.g.append(put(dev(synth.normal_f32((n,), 0.1, seed + 7 * k + 1)).to(gdt)))
            if small:
                self.m.append(tuple(put(t) for t in zeros8(n)))
                self.v.append(tuple(put(t) for t in zeros8(n)))
            else:
                self.m.append(put(torch.zeros(n, device="cuda")))
                self.v.append(put(torch.zeros(n, device="cuda")))
            self.copy.append(put(torch.zeros(n, dtype=BF16, device="cuda")) if copy else None)
            self.wd.append(wd)
        self.plan = R().wbmm_adamw_plan(self.p, self.g, self.m, self.v, copies=self.copy,
                                        weight_decay=self.wd)

    @staticmethod
    def _np(t):
        return tuple(x.cpu().numpy() for x in t) if isinstance(t, tuple) else t.cpu().numpy()

    def host(self):
        return [(self._np(p), g.float().cpu().numpy(), self._np(m), self._np(v))
                for p, g, m, v in zip(self.p, self.g, self.m, self.v)]

    def new_gradients(self, seed):
        for k, g in enumerate(self.g):
            g.copy_(dev(synth.normal_f32((g.numel(),), 0.1, seed + k)))


def same(a, b):
    if isinstance(a, tuple):
        return all(same(x, y) for x, y in zip(a, b))
    return np.array_equal(a, b) or (a.dtype == np.float32 and np.array_equal(a.view(np.uint32),
                                                                             b.view(np.uint32)))


SPEC = [(n, gdt, small, copy, 0.1 if n % 2 else 0.0)
        for n, gdt, small, copy in [(1, F32, True, True), (2, BF16, False, False), (31, F32, True, False),
                                    (32, BF16, True, True), (33, F32, False, True), (97, BF16, True, False),
                                    (4095, F32, True, True), (4096, F32, False, True), (4097, BF16, True, False),
                                    (12289, F32, True, False), (20000, BF16, False, True)]]


@pytest.mark.parametrize("shift", [0, 1])
def test_steps_equal_the_oracle(shift):
    s = Model(SPEC, 1, shift)
    for step in (1, 2, 3):
        before = s.host()
        R().wbmm_adamw_step(s.plan, lr=KW["lr"], betas=(KW["b1"], KW["b2"]), eps=KW["eps"], step=step, seed=77)
        for k, ((p, g, m, v), (p1, _, m1, v1)) in enumerate(zip(before, s.host())):
            wp, wm, wv = K.adamw(p, g, m, v, wd=s.wd[k], step=step, tensor=k, seed=77, **KW)
            assert same(p1, wp) and same(m1, wm) and same(v1, wv), (k, step)
            if s.copy[k] is not None:
                assert torch.equal(s.copy[k], s.p[k].to(BF16))
        s.new_gradients(50 * step)


def test_large_seed_and_step():
    s = Model([(100, F32, True, False, 0.0)], 3)
    (p, g, m, v), seed, step = s.host()[0], (0xfedcba98 << 32) | 0x76543210, 2 ** 31 - 1
    R().wbmm_adamw_step(s.plan, lr=KW["lr"], betas=(KW["b1"], KW["b2"]), eps=KW["eps"], step=step, seed=seed)
    wp, wm, wv = K.adamw(p, g, m, v, wd=0.0, step=step, seed=seed, **KW)
    p1, _, m1, v1 = s.host()[0]
    assert same(p1, wp) and same(m1, wm) and same(v1, wv)


def test_against_64_bits():
    """20 steps with fp32 states: an operation rounds by half a step, a step of p has about 10 of them on
    the update (at most 3 lr here) and 2 on p: 2^-24 (30 lr + 2 |p|) a step; m and v contract."""
    s = Model([(3000, F32, False, False, 0.1)], 5)
    p, _, m, v = (x.astype(np.float64) for x in s.host()[0])
    for step in range(1, 21):
        g = s.host()[0][1].astype(np.float64)
        R().wbmm_adamw_step(s.plan, lr=KW["lr"], betas=(KW["b1"], KW["b2"]), eps=KW["eps"], step=step)
        p, m, v = K.adamw64(p, g, m, v, wd=0.1, step=step, **KW)
        got = s.host()[0]
        assert np.all(np.abs(got[0] - p) <= step * 2.0 ** -24 * (60 * KW["lr"] + 2 * np.abs(p)))
        s.new_gradients(step * 11)


def test_factors_and_step_on_the_device():
    a, b = Model(SPEC, 9), Model(SPEC, 9)
    lr, gr = torch.full((1,), 0.5, device="cuda"), torch.full((1,), 0.25, device="cuda")
    count = torch.ones(1, dtype=torch.int32, device="cuda")
    for step in (1, 2):
        before = a.host()
        R().wbmm_adamw_step(a.plan, lr=0.02, betas=(0.9, 0.99), step=step, lr_factor=lr, grad_factor=gr, seed=5)
        R().wbmm_adamw_step(b.plan, lr=0.02, betas=(0.9, 0.99), step=count, lr_factor=lr, grad_factor=gr, seed=5)
        count += 1
        for k, (x, y, (p, g, m, v)) in enumerate(zip(a.host(), b.host(), before)):
            wp, wm, wv = K.adamw(p, g, m, v, lr=0.02, b1=0.9, b2=0.99, eps=1e-8, wd=a.wd[k], step=step, tensor=k,
                                 seed=5, lr_factor=0.5, grad_factor=0.25)
            assert same(x[0], wp) and same(x[2], wm) and same(x[3], wv)
            # the device forms beta^t by its own power: its factors may be off by a last bit
            assert np.all(np.abs(y[0] - x[0]) <= 2.0 ** -23 * (np.abs(x[0]) + 0.1))


def test_replayed_counting_on_the_device():
    a, b = Model(SPEC, 13), Model(SPEC, 13)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    other = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(s, c):
        c.add_(1)
        R().wbmm_adamw_step(s.plan, lr=0.02, step=c, seed=5)

    step(a, count)
    step(b, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, count)
    for _ in range(3):
        step(b, other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(x[0], y[0]) and same(x[2], y[2]) and same(x[3], y[3]) for x, y in zip(a.host(), b.host()))
    assert int(count) == 4


def test_nan_and_infinite_gradients():
    """fp32 states: the element alone; 8-bit states: its group's states, no other parameter."""
    for small in (False, True):
        s = Model([(100, F32, small, True, 0.1)], 21)
        clean = Model([(100, F32, small, True, 0.1)], 21)
        s.g[0][40], s.g[0][70] = float("nan"), float("inf")
        for x in (s, clean):
            R().wbmm_adamw_step(x.plan, lr=0.01, step=1, seed=3)
        p, q = s.p[0], clean.p[0]
        hit = torch.zeros(100, dtype=torch.bool, device="cuda")
        hit[[40, 70]] = True
        assert torch.equal(p[~hit], q[~hit]) and p[40].isnan() and p[70].isnan()
        if small:
            for st, cl in ((s.m[0], clean.m[0]), (s.v[0], clean.v[0])):
                assert [int(x) for x in st[1].cpu()][1:3] == [255, 255]
                assert torch.equal(st[0][:32], cl[0][:32]) and torch.equal(st[0][96:], cl[0][96:])
                assert torch.equal(st[1][[0, 3]], cl[1][[0, 3]])


def test_eight_bit_states_follow():
    """200 steps of constant gradients, b2 = 0.999. m and v tend to g and g^2; nearest rounding would leave the
    root where it first stood, at 3 % of g. An element's rounding is 2^-4 of itself at most; 200 of them add
    up to a random walk of 2^-4 sqrt(200) / 2 = 0.44, the mean of 4096 elements to 0.7 %, three of which are
    2 %. The rounding is right on average for the root r, not for its square: a step d of the root against
    a spacing s of the codes goes up by s in d / s of the cases, which adds the variance d s to r^2, on top of
    2 r d. As s <= r / 8, r^2 grows by 1 to 1 + 1/16 of the recurrence, the root is up to 3.1 % above it."""
    n = 4096
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
    m, v = zeros8(n), zeros8(n)
    plan = R().wbmm_adamw_plan([p], [g], [m], [v])
    for t in range(1, 201):
        R().wbmm_adamw_step(plan, lr=1e-3, betas=(0.9, 0.999), step=t, seed=11)
    root = R().wbmm_ckpt_unpack(*v, fmt="e4m3").double().square().mean().sqrt()
    want = 0.5 * np.sqrt(1 - 0.999 ** 200)
    assert -0.02 < float(root) / want - 1 < 0.031 + 0.02
    assert abs(float(R().wbmm_ckpt_unpack(*m, fmt="e4m3").mean()) / 0.5 - 1) < 0.02


def test_nothing_else_is_written():
    spec = [(n, F32, small, True, 0.0) for n in (5, 4097, 9000) for small in (False, True)]
    pad, keep = 64, []

    def guarded(n, dt):
        flat = torch.full((n + 2 * pad,), 77 if dt == U8 else 3.0, dtype=dt, device="cuda")
        keep.append((flat, n))
        flat[pad:pad + n] = 0
        return flat[pad:pad + n]

    p = [guarded(n, F32) for n, *_ in spec]
    g = [torch.ones(n, device="cuda") for n, *_ in spec]
    st = [[(guarded(n, U8), guarded(-(-n // 32), U8)) if small else guarded(n, F32) for n, _, small, *_ in spec]
          for _ in range(2)]
    copies = [guarded(n, BF16) for n, *_ in spec]
    plan = R().wbmm_adamw_plan(p, g, st[0], st[1], copies=copies)
    R().wbmm_adamw_step(plan, lr=0.1, step=1)
    assert all(torch.all(x != 0) for x in p)
    for flat, n in keep:
        fill = 77 if flat.dtype == U8 else 3.0
        assert torch.all(flat[:pad] == fill) and torch.all(flat[pad + n:] == fill)


def test_a_table_of_other_counts_is_left_alone():
    s = Model(SPEC, 30)
    want = s.host()
    lib, stream = R()._lib(), torch.cuda.current_stream().cuda_stream
    for count, chunks in ((s.plan.count, s.plan.chunks + 1), (s.plan.count - 1, s.plan.chunks)):
        assert lib.wbmm_adamw_step(s.plan.ptr, count, chunks, 0.1, 0.9, 0.999, 1e-8, 1, None, None, None, 0,
                                   stream) == 0
    torch.cuda.synchronize()
    assert all(same(a[0], b[0]) and same(a[2], b[2]) for a, b in zip(want, s.host()))


def test_a_tensor_past_32_bits():
    """2^30 + 5000 parameters, bf16 gradients, 8-bit states: the last ones are those of a small tensor but for
    their counters, which the fp32 part does not use."""
    n, k = (1 << 30) + 5000, 5000
    p, g = torch.ones(n, device="cuda"), torch.ones(n, dtype=BF16, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[-k:] = dev(synth.normal_f32((k,), 1.0, 2)).to(BF16)
    small = [t[-k:].clone() for t in (p, g, m, v)]
    a = R().wbmm_adamw_plan([p], [g], [m], [v])
    b = R().wbmm_adamw_plan([small[0]], [small[1]], [small[2]], [small[3]])
    for plan in (a, b):
        R().wbmm_adamw_step(plan, lr=0.1, step=1)
    assert all(torch.equal(x[-k:], y) for x, y in zip((p, m, v), (small[0], small[2], small[3])))
    assert torch.all(p[:: 1 << 20][:1000] == p[0])


def test_refused_plans():
    M = R()
    t = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    p, g, m, v = t(64), t(64), t(64), t(64)
    bad = [([p, p], [g, g], [m, t(64)], [v, t(64)]), ([p], [p], [m], [v]), ([p], [g], [m], [m]),
           ([p[:33], p[32:]], [t(33), t(32)], [t(33), t(32)], [t(33), t(32)]), ([], [], [], []),
           ([p], [g], [m], []), ([p], [g[:3]], [m], [v]), ([p], [g.half()], [m], [v]),
           ([p], [g], [zeros8(64)], [v]), ([p.cpu()], [g], [m], [v]), ([p], [g], [(m, m)], [(v, v)])]
    for args in bad:
        with pytest.raises(M.WbmmError):
            M.wbmm_adamw_plan(*args)
    M.wbmm_adamw_plan([p, t(64)], [g, g], [m, t(64)], [v, t(64)])     # one gradient for two tensors
    plan = M.wbmm_adamw_plan([p], [g], [m], [v])
    for kw in (dict(step=0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0),
               dict(step=torch.ones(2, dtype=torch.int32, device="cuda")), dict(lr_factor=torch.ones(1))):
        with pytest.raises(M.WbmmError):
            M.wbmm_adamw_step(plan, **{"lr": 0.1, **kw})


def test_eight_bit_states_past_32_bits():
    """2^32 + 5000 parameters with bf16 gradients and 8-bit states: the first 4000 and the last 5000, which lie from
    element 2^32 on, equal the oracle after two steps, codes, scales and the counters of the random words."""
    n, k = (1 << 32) + 5000, 5000
    p, g = torch.ones(n, device="cuda"), torch.ones(n, dtype=BF16, device="cuda")
    m, v = zeros8(n), zeros8(n)
    for part in (slice(0, 4000), slice(n - k, n)):
        g[part] = dev(synth.normal_f32((part.stop - part.start,), 1.0, 2)).to(BF16)
    plan = R().wbmm_adamw_plan([p], [g], [m], [v], weight_decay=0.1)

    def host(part):
        groups = slice(part.start // 32, -(-part.stop // 32))
        get = lambda t: t.cpu().numpy()  # noqa: E731
        return (get(p[part]), g[part].float().cpu().numpy(), *((get(c[part]), get(s[groups])) for c, s in (m, v)))

    for step in (1, 2):
        before = [host(part) for part in (slice(0, 4000), slice(n - k, n))]
        R().wbmm_adamw_step(plan, lr=KW["lr"], betas=(KW["b1"], KW["b2"]), eps=KW["eps"], step=step, seed=77)
        for part, (p0, g0, m0, v0) in zip((slice(0, 4000), slice(n - k, n)), before):
            wp, wm, wv = K.adamw(p0, g0, m0, v0, wd=0.1, step=step, seed=77, first=part.start, **KW)
            p1, _, m1, v1 = host(part)
            assert same(p1, wp) and same(m1, wm) and same(v1, wv), (part, step)
        if step == 1:      # equal parameters, gradients and states; from then on the states' roundings differ
            assert torch.all(p[1 << 20::1 << 20] == p[1 << 20])
