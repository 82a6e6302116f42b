"""The recurrence's layout rules, compiled for the host alone: what they choose for a call has to be a
launch that the runtime takes and that the kernels assume, over the sizes that the calls admit."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "receptive_field_spatial_amd", "csrc")

SHIM = r"""
#include "wbmm_scanplan.cpp"
extern "C" void plan(int64_t o, int64_t l, int64_t i, int bf16, int kind, int ck, int64_t* r) {
  const wbmm::ScanPlan p = wbmm::scan_plan(o, l, i, bf16, kind, ck);
  const int64_t v[] = {p.rows, p.wide, p.self, p.cw, p.lanes, p.waves, p.segs, p.seg_len, p.fine,
                       wbmm::scan_col_waves(kind != 0, ck, p.wide), wbmm::scan_map_waves(ck && kind == 0)};
  for (int k = 0; k < 11; ++k) r[k] = v[k];
}
"""
NAMES = "rows wide self cw lanes waves segs seg_len fine col_waves map_waves".split()
K, E = 16, 8   # steps per lane and tile, columns and rows


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "plan.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"), "-o", so],
                   check=True)
    fn = ctypes.CDLL(so).plan
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p]

    def call(o, l, i, bf16, kind, ck):
        r = (ctypes.c_int64 * 11)()
        fn(o, l, i, bf16, kind, ck, r)
        return dict(zip(NAMES, r))

    return call


def check(p, o, l, i, kind):
    cols = o * i
    threads = 64 * p["waves"]
    assert 1 <= p["waves"] <= 16
    if p["lanes"] < 64:
        assert p["rows"] and p["segs"] == 1 and p["self"] and l <= p["lanes"] * E
        per = p["waves"] * (64 // p["lanes"])
        assert -(-cols // per) * threads < 1 << 32
        return
    if p["rows"]:
        groups, piece, map_waves = cols, 64 * E, p["waves"]
    else:
        assert p["waves"] <= p["col_waves"] and p["cw"] in (1, 2, 4, 8, 16, 32, 64)
        groups, piece, map_waves = -(-cols // p["cw"]), 64 // p["cw"] * K, p["map_waves"]
        if kind and p["cw"] == 64:
            assert p["waves"] % 2 == 0   # waves pair up for the kept states
    # a launch has fewer than 2^32 threads along x, and no more than 65535 workgroups along y
    assert groups * threads < 1 << 32
    assert (p["segs"] - 1) * p["fine"] <= 65535
    tile = p["waves"] * piece
    assert p["seg_len"] % tile == 0
    assert p["segs"] * p["seg_len"] >= l > (p["segs"] - 1) * p["seg_len"]
    if p["segs"] > 1:
        assert groups * 64 * map_waves < 1 << 32
        assert p["seg_len"] % p["fine"] == 0 and p["seg_len"] // p["fine"] % (map_waves * piece) == 0
        assert not p["self"]
    if kind == 2 and p["self"]:
        assert l <= tile   # one tile holds the axis


def every(plan, o, l, i):
    for bf16 in (0, 1):
        for kind in (0, 1, 2):
            for ck in (0, 1):
                try:
                    check(plan(o, l, i, bf16, kind, ck), o, l, i, kind)
                except AssertionError as e:
                    raise AssertionError((o, l, i, bf16, kind, ck, plan(o, l, i, bf16, kind, ck))) from e


TOP = (1 << 26) - 1   # columns, at most


@pytest.mark.parametrize("o,l,i", [
    (1 << 25, 513, 1), (1 << 25, 600, 1), (1 << 25, 1024, 1), (22500000, 1100, 1), (TOP, 700, 1),
    (TOP, 4096, 1), (TOP, 256, 1), (TOP, 257, 1), (TOP, 1, 1), (1 << 23, 8000, 1), (1 << 22, 8192, 1),
    (1, 1 << 30, 1), (1, 1 << 30, 200), (TOP // 3, 1000, 3), (1, 4096, TOP), (1 << 20, 3000, 60),
])
def test_largest_launches(plan, o, l, i):
    every(plan, o, l, i)


def test_small_sizes(plan):
    for o in (1, 2, 3, 64, 127, 128, 129, 300, 1025):
        for i in (1, 2, 3, 4, 7, 8, 16, 31, 33, 63, 64, 65, 200):
            for l in (1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 511, 512, 513, 1024, 1025, 8193):
                every(plan, o, l, i)


def test_random_sizes(plan):
    rng = random.Random(3)
    size = lambda top: max(1, min(top, int(2 ** rng.uniform(0, top.bit_length()))))
    n = 0
    while n < 4000:
        o, i, l = size(TOP), rng.choice((1, size(4000))), size(1 << 30)
        if o * i <= TOP and o * i * l <= 1 << 38:
            every(plan, o, l, i)
            n += 1
