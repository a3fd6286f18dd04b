"""Host side of the microscaled operators: sizes and refusals, checked before
anything reaches a GPU."""
import numpy as np
import pytest

import mx_util as mx
import sparse_mixture_experts_histogram_b200 as moe
from sparse_mixture_experts_histogram_b200 import build

FAKE = 1 << 20  # an aligned address that is never dereferenced
ROOM = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


def test_scale_pitch(lib):
    for cols, want in ((32, 16), (512, 16), (544, 32), (4096, 128), (1408, 48), (0, 0), (-32, 0), (48, 0)):
        assert moe.moe_mx_scale_pitch(cols) == want


def test_constants_are_the_headers(lib):
    import os
    h = open(os.path.join(build.INCLUDE, "moe.h")).read()
    for name, v in (("MOE_TYPE_BF16", moe.TYPE_BF16), ("MOE_TYPE_FP16", moe.TYPE_FP16), ("MOE_TYPE_FP32", moe.TYPE_FP32),
                    ("MOE_MX_E4M3", moe.MX_E4M3), ("MOE_MX_E2M1", moe.MX_E2M1)):
        assert f"#define {name} {v}\n" in h


def test_workspace_sizes(lib):
    for S, E, N in ((1, 1, 8), (2, 8, 4096), (8192, 8, 14336), (1 << 20, 256, 65536)):
        assert 256 <= moe.moe_mx_workspace_size(S, E, N) <= 64 << 20
    for bad in ((0, 1, 128), (1, 0, 128), (1, 257, 128), (1, 1, 12), (1, 1, 65544), ((1 << 27) + 1, 1, 128)):
        assert moe.moe_mx_workspace_size(*bad) == 0
    assert moe.moe_forward_mx_workspace_size(16, 256, 8, 512, 2) > 0
    assert moe.moe_forward_mx_workspace_size(16, 250, 8, 512, 2) == 0


GOOD = dict(rows=4, cols=64, type=0, x=FAKE, stride=64, fmt=1, q=FAKE, s=FAKE, hat=FAKE)


@pytest.mark.parametrize("change,want", [
    (dict(rows=0), 1), (dict(cols=0), 1), (dict(type=3), 1), (dict(type=-1), 1), (dict(fmt=2), 1),
    (dict(cols=48), 2), (dict(rows=(1 << 34) // 64 + 1), 2), (dict(cols=(1 << 20) + 32), 2),
    (dict(stride=32), 1), (dict(stride=65), 1), (dict(stride=-64), 1), (dict(x=None), 1),
    (dict(x=FAKE + 2), 1), (dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(s=None), 1),
    (dict(s=FAKE + 1), 1), (dict(hat=FAKE + 4), 1),
])
def test_quantize_refusals(lib, change, want):
    a = {**GOOD, **change}
    assert lib.moe_mx_quantize(a["rows"], a["cols"], a["type"], a["x"], a["stride"], a["fmt"],
                               a["q"], a["s"], a["hat"], None) == want


NORM = dict(T=4, d=64, type=0, h=FAKE, hs=64, dt=2, delta=FAKE, ds=64, w=FAKE, eps=1e-6,
            ho=FAKE + 4096, y=FAKE + 8192, q=FAKE, s=FAKE)


@pytest.mark.parametrize("change,want", [
    (dict(T=0), 1), (dict(d=0), 1), (dict(d=48), 2), (dict(d=16416), 2), (dict(T=(1 << 24) + 1), 2),
    (dict(type=3), 1), (dict(dt=1), 1), (dict(type=2, dt=0), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(h=None), 1), (dict(h=FAKE + 4), 1),
    (dict(hs=60), 1), (dict(hs=68), 1), (dict(ds=66), 1), (dict(delta=FAKE + 8), 1), (dict(w=None), 1),
    (dict(w=FAKE + 2), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(ho=None, y=None, q=None, s=None), 1),
    (dict(ho=FAKE + 2), 1), (dict(y=FAKE + 2), 1), (dict(q=FAKE + 2), 1), (dict(s=FAKE + 2), 1),
    (dict(ho=FAKE, hs=128), 1),
])
def test_rmsnorm_refusals(lib, change, want):
    a = {**NORM, **change}
    assert lib.moe_rmsnorm(a["T"], a["d"], a["type"], a["h"], a["hs"], a["dt"], a["delta"], a["ds"],
                           a["w"], a["eps"], a["ho"], a["y"], a["q"], a["s"], None) == want


PROD = dict(S=4, K=256, E=2, N=64, fmt=0, x=FAKE, xs=FAKE, off=FAKE, W=FAKE, Ws=FAKE, yt=0, y=FAKE,
            ws=FAKE, room=ROOM)


@pytest.mark.parametrize("change,want", [
    (dict(S=0), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(N=0), 1), (dict(K=192), 2), (dict(N=60), 2),
    (dict(E=257), 2), (dict(K=65664), 2), (dict(N=65544), 2), (dict(S=(1 << 27) + 1), 2), (dict(fmt=2), 1),
    (dict(yt=1), 1), (dict(x=None), 1), (dict(xs=None), 1), (dict(W=None), 1), (dict(Ws=None), 1),
    (dict(y=None), 1), (dict(y=FAKE + 8), 1), (dict(W=FAKE + 8), 1), (dict(off=None), 1), (dict(off=FAKE + 4), 1),
    (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(room=64), 3),
])
def test_product_refusals(lib, change, want):
    a = {**PROD, **change}
    assert lib.moe_mx_product(a["S"], a["K"], a["E"], a["N"], a["fmt"], a["x"], a["xs"], a["off"], a["W"],
                              a["Ws"], a["yt"], a["y"], a["ws"], a["room"], None) == want


GATED = dict(S=4, d=256, E=2, f=128, fmt=0, x=FAKE, xs=FAKE, off=FAKE, W1=FAKE, s1=FAKE, W3=FAKE, s3=FAKE,
             act=0, h=None, hq=FAKE, hs=FAKE, ws=FAKE, room=ROOM)


@pytest.mark.parametrize("change,want", [
    (dict(S=0), 1), (dict(d=192), 2), (dict(f=64), 2), (dict(act=2), 1), (dict(act=-1), 1), (dict(fmt=-1), 1),
    (dict(W1=None), 1), (dict(s1=None), 1), (dict(W3=None), 1), (dict(s3=None), 1), (dict(h=FAKE), 1),
    (dict(hq=None), 1), (dict(hs=None), 1), (dict(hq=None, hs=None), 1), (dict(h=FAKE + 2, hq=None, hs=None), 1),
    (dict(hs=FAKE + 4), 1), (dict(ws=FAKE + 16), 1), (dict(room=64), 3), (dict(off=None), 1),
])
def test_gated_refusals(lib, change, want):
    a = {**GATED, **change}
    assert lib.moe_mx_gated(a["S"], a["d"], a["E"], a["f"], a["fmt"], a["x"], a["xs"], a["off"], a["W1"], a["s1"],
                            a["W3"], a["s3"], a["act"], a["h"], a["hq"], a["hs"], a["ws"], a["room"], None) == want


FWD = dict(T=4, d=256, E=8, f=512, k=2, h=FAKE, delta=FAKE, w=FAKE, eps=1e-6, ho=FAKE, Wg=FAKE, bias=FAKE,
           W1=FAKE, s1=FAKE, W3=FAKE, s3=FAKE, W2=FAKE, s2=FAKE, out=FAKE, ws=FAKE, room=ROOM)


@pytest.mark.parametrize("change,want", [
    (dict(T=0), 1), (dict(k=9), 1), (dict(d=200), 2), (dict(f=200), 2), (dict(eps=0.0), 1), (dict(h=None), 1),
    (dict(w=None), 1), (dict(Wg=None), 1), (dict(W1=None), 1), (dict(s1=FAKE + 8), 1), (dict(W3=None), 1),
    (dict(s3=None), 1), (dict(W2=None), 1), (dict(s2=None), 1), (dict(out=None), 1), (dict(delta=FAKE + 4), 1),
    (dict(ho=FAKE + 4), 1), (dict(bias=FAKE + 4), 1), (dict(ws=FAKE + 16), 1), (dict(room=4096), 3),
])
def test_forward_refusals(lib, change, want):
    a = {**FWD, **change}
    assert lib.moe_forward_mx(a["T"], a["d"], a["E"], a["f"], a["k"], a["h"], a["delta"], a["w"], a["eps"], a["ho"],
                              a["Wg"], a["bias"], a["W1"], a["s1"], a["W3"], a["s3"], a["W2"], a["s2"], a["out"],
                              a["ws"], a["room"], None) == want


def test_the_formats_in_64_bits():
    """The tests' own restatement of the formats, on values worked out by hand."""
    assert mx.grid(mx.E4M3)[-1] == 448 and mx.grid(mx.E4M3)[1] == 2.0 ** -9 and len(mx.grid(mx.E4M3)) == 127
    x = np.zeros((1, 32))
    x[0, :8] = (6, -5, 2.5, 3.5, 0.25, 0.75, -0.2, 1.75)   # ties go to the even code
    c, s = mx.quantize(x, mx.E2M1)
    assert s[0, 0] == 127 and (mx.values(c, s, mx.E2M1)[0, :8] == (6, -4, 2, 4, 0, 1, 0, 2)).all()
    assert mx.scale_code([0.0, 6.0, 6.0001, 12.0, 3.0, np.inf, np.nan], mx.E2M1).tolist() == [0, 127, 128, 128, 126, 255, 255]
    assert mx.scale_code([448.0, 449.0, 1e-300], mx.E4M3).tolist() == [127, 128, 0]
    assert (mx.unpack(mx.pack(c, mx.E2M1), mx.E2M1) == c).all()
