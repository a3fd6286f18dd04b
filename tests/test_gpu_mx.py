"""The microscaled operators on the GPU against their formulas in 64 bits.

Tolerances: a rounding is off by at most half a step (eps / 2 relative).  A
sum of K products in fp32, whatever its order, is off by at most K 2^-23 of the
sum of the magnitudes (2^-23, not 2^-24, an addition: the tensor cores may cut
off instead of rounding).
"""
import numpy as np
import pytest
import torch

import mx_util as mx
import sparse_mixture_experts_histogram_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def byte(*shape, fill=0xA5):
    return torch.full(shape, fill, dtype=torch.uint8, device=DEV)


def f64(t):
    return t.double().cpu().numpy()


def ws_for(S, E, N):
    return byte(moe.moe_mx_workspace_size(S, E, N), fill=0xFF)


def ok(ws):
    st, code = moe.moe_get_device_error(ws)
    assert st == 0, f"device error word {code:#x}"


# ------------------------------------------------------------------ quantise

@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("rows,cols,extra", [(1, 32, 0), (3, 96, 32), (17, 512, 0), (33, 544, 8), (130, 1408, 64), (1, 16416, 0), (5000, 64, 0)])
def test_quantize_is_exact(type, fmt, rows, cols, extra):
    t = mx.TORCH[type]
    g = torch.Generator(device=DEV).manual_seed(rows * cols + type)
    big = torch.randn(rows, cols + extra, generator=g, device=DEV)
    big *= torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g, device=DEV).float())
    big = big.to(t)
    x = big[:, :cols]
    q, s = byte(rows, cols if fmt == mx.E4M3 else cols // 2), byte(rows, mx.pitch(cols))
    hat = torch.empty(rows, cols, dtype=t, device=DEV)
    moe.moe_mx_quantize(rows, cols, type, x, cols + extra, fmt, q, s, hat)
    c, sc = mx.quantize(f64(x), fmt)
    assert (s.cpu().numpy() == mx.scale_rows(sc)).all()
    assert (q.cpu().numpy() == mx.pack(c, fmt)).all()
    want = torch.from_numpy(mx.values(c, sc, fmt)).to(t)
    assert torch.equal(hat.cpu(), want)
    q2, s2 = byte(*q.shape), byte(*s.shape)
    moe.moe_mx_quantize(rows, cols, type, x, cols + extra, fmt, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
def test_quantize_borders(fmt):
    """Every midpoint of the format and its neighbours, powers of two around
    the scale's borders, zeros, subnormals, infinities, NaN."""
    g = mx.grid(fmt)
    mid = (g[1:] + g[:-1]) / 2
    pts = np.concatenate([mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 1e9), g])
    pts = np.concatenate([pts, -pts])
    pts = np.concatenate([pts, np.zeros(-len(pts) % 31)])
    rows = [np.concatenate([[mx.MOST[fmt]], r]) for r in pts.reshape(-1, 31)]       # scale 1
    rows += [np.full(32, mx.MOST[fmt] * 2.0 ** e) for e in (-149, -140, -127, -126, -60, 0, 60, 118)]
    rows += [np.full(32, np.nextafter(np.float32(mx.MOST[fmt] * 2.0 ** e), np.float32(np.inf))) for e in (-127, -60, 0, 60)]
    rows += [np.zeros(32), np.full(32, -0.0), np.full(32, 2.0 ** -149), np.full(32, np.finfo(np.float32).max)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(32)
        r[17] = bad
        rows.append(r)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(DEV)
    n = len(rows)
    q, s, hat = byte(n, 32 if fmt == mx.E4M3 else 16), byte(n, 16), torch.empty_like(x)
    moe.moe_mx_quantize(n, 32, 2, x, 32, fmt, q, s, hat)
    c, sc = mx.quantize(f64(x), fmt)
    assert (s.cpu().numpy() == mx.scale_rows(sc)).all()
    assert (q.cpu().numpy() == mx.pack(c, fmt)).all()
    assert np.array_equal(hat.cpu().numpy(), mx.values(c, sc, fmt).astype(np.float32), equal_nan=True)


# ---------------------------------------------------------------------- norm

@pytest.mark.parametrize("type,dt", [(0, None), (0, 0), (0, 2), (1, 1), (1, 2), (2, None), (2, 2)])
@pytest.mark.parametrize("T,d,extra", [(1, 32, 0), (3, 96, 32), (130, 512, 0), (7, 1408, 8), (2, 4096, 0), (5, 7168, 64), (2, 8224, 0), (3, 16384, 0)])
def test_rmsnorm_matches_formula(type, dt, T, d, extra):
    t = mx.TORCH[type]
    g = torch.Generator(device=DEV).manual_seed(T * d + type)
    h = (3 * torch.randn(T, d + extra, generator=g, device=DEV)).to(t)
    delta = None if dt is None else torch.randn(T, d + extra, generator=g, device=DEV).to(mx.TORCH[dt])
    w = (1 + torch.randn(d, generator=g, device=DEV)).to(t)
    ho, y = torch.empty(T, d, dtype=t, device=DEV), torch.empty(T, d, dtype=t, device=DEV)
    q, s = byte(T, d), byte(T, mx.pitch(d))
    eps = 1e-5
    moe.moe_rmsnorm(T, d, type, h, d + extra, type if dt is None else dt, delta, d + extra, w, eps, ho, y, q, s)
    sums = h[:, :d].float()
    if delta is not None:
        sums = sums + delta[:, :d].float()
    assert torch.equal(ho, sums.to(t))
    v = f64(ho)
    n = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))) * f64(w)
    # the factor, its two products: three roundings of 2^-24
    slack = 4 * 2.0 ** -24
    assert (np.abs(f64(y) - n) <= (HALF[t] + slack) * np.abs(n) + TINY[t]).all()
    pad = s[:, d // 32:]
    assert pad.numel() == 0 or int(pad.max()) == 0
    assert mx.code_error(q.cpu().numpy().astype(np.int64), s[:, :d // 32].cpu().numpy().astype(np.int64), n, slack) <= 0
    # each output alone gives the same
    y2, q2, s2 = torch.empty_like(y), byte(T, d), byte(T, mx.pitch(d))
    args = (T, d, type, h, d + extra, type if dt is None else dt, delta, d + extra, w, eps)
    moe.moe_rmsnorm(*args, None, y2, None, None)
    moe.moe_rmsnorm(*args, None, None, q2, s2)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("type,size", [(0, 3e30), (0, 1e-25), (0, 3e38), (1, 6e4), (1, 1e-7)])
def test_rmsnorm_of_16_bit_extremes(type, size):
    """Squares that leave fp32's range, above and below."""
    t, T, d = mx.TORCH[type], 3, 1376
    h = (torch.randn(T, d, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).clamp(-1, 1) * size).to(t)
    w, y, eps = torch.ones(d, dtype=t, device=DEV), torch.empty(T, d, dtype=t, device=DEV), 1e-38
    moe.moe_rmsnorm(T, d, type, h, d, type, None, d, w, eps, None, y, None, None)
    v = f64(h)
    n = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    assert (np.abs(f64(y) - n) <= (HALF[t] + 4 * 2.0 ** -24) * np.abs(n) + TINY[t]).all()


def test_rmsnorm_in_place_and_extremes():
    d = 256
    h = torch.zeros(6, d, device=DEV)
    h[1] = 1e30
    h[2] = 1e-30
    h[3, 5] = float("nan")
    h[4, 5] = float("inf")
    h[5, 0] = torch.finfo(torch.float32).max
    w = torch.ones(d, device=DEV)
    y, q, s = torch.empty_like(h), byte(6, d), byte(6, 16)
    kept = h.clone()
    moe.moe_rmsnorm(6, d, 2, h, d, 2, torch.zeros_like(h), d, w, 1e-6, h, y, q, s)
    assert torch.equal(h.nan_to_num(7.0), kept.nan_to_num(7.0))
    assert (y[0] == 0).all() and int(s[0].max()) == 0
    assert torch.allclose(y[1], torch.ones(d, device=DEV), rtol=4 * 2.0 ** -24, atol=0)   # squares leave fp32
    assert torch.allclose(y[2], torch.full((d,), 1e-27, device=DEV), rtol=1e-6, atol=0)
    assert y[3].isnan().all() and (s[3, :8] == 255).all() and (q[3] == 0).all()
    # inf / inf is NaN, and 0 of the others: their block reads back as zeros
    assert y[4, 5].isnan() and (y[4, :5] == 0).all() and s[4, 0] == 255 and s[4, 1] == 0
    assert abs(y[5, 0].item() - 16.0) < 1e-5


# ------------------------------------------------------------- the products

def segments(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32), device=DEV)


def product_ref(x, W, sizes):
    """(y, sum of magnitudes) in 64 bits."""
    y, a, r = [], [], 0
    for e, n in enumerate(sizes):
        y.append(x[r:r + n] @ W[e].T)
        a.append(np.abs(x[r:r + n]) @ np.abs(W[e]).T)
        r += n
    return np.concatenate(y), np.concatenate(a)


SIZES = [
    ([1], 128, 8), ([3], 256, 136), ([2, 0, 1], 128, 1000), ([0, 5, 0, 0], 384, 264),
    ([37, 0, 128, 1, 200, 64], 640, 392), ([191, 193, 192], 512, 520), ([700, 16], 1408, 264),
    ([1] * 40, 256, 256), ([2, 1], 14336, 512), ([17] * 9, 2048, 640),
    ([80], 384, 264), ([70, 60], 640, 136), ([95], 128, 16),
    ([5, 4], 640, 72), ([4, 3], 384, 24), ([20], 1152, 40), ([3] * 5, 896, 264), ([7, 9, 1], 1536, 520),
    ([1], 4096, 256), ([0, 3], 3584, 8), ([1] * 75, 3200, 256),   # cut units of fewer chunks than there are CTA pairs
]


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("sizes,K,N", SIZES)
@pytest.mark.parametrize("yt", [0, 2])
def test_product_matches_formula(fmt, sizes, K, N, yt):
    rng = np.random.default_rng(len(sizes) + K + N)
    E, R = len(sizes), sum(sizes)
    S = R + 3                                      # rows behind the last segment
    x = mx.Matrix(rng, (S, K), fmt)
    x.s[R:] = 0xFF                                 # a NaN there must reach nothing
    W = mx.Matrix(rng, (E, N, K), mx.E2M1, K ** -0.5)
    t = mx.TORCH[yt]
    y = torch.full((S, N), 7.0, dtype=t, device=DEV)
    ws = ws_for(S, E, N)
    moe.moe_mx_product(S, K, E, N, fmt, x.q, x.s, segments(sizes), W.q, W.s, yt, y, ws)
    ok(ws)
    assert (y[R:] == 7).all()
    ref, mag = product_ref(x.v, W.v, sizes)
    err = np.abs(f64(y[:R]) - ref)
    assert (err <= K * 2.0 ** -23 * mag * (1 + HALF[t]) + HALF[t] * np.abs(ref)).all()
    # again, on the same inputs: the same bits
    y2 = torch.full((S, N), 7.0, dtype=t, device=DEV)
    moe.moe_mx_product(S, K, E, N, fmt, x.q, x.s, segments(sizes), W.q, W.s, yt, y2, ws)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("S,K,N", [(1, 512, 256), (5, 128, 24), (300, 896, 328), (8, 4096, 4096)])
def test_product_without_segments(fmt, S, K, N):
    rng = np.random.default_rng(S)
    x, W = mx.Matrix(rng, (S, K), fmt), mx.Matrix(rng, (1, N, K), mx.E2M1)
    y = torch.empty(S, N, device=DEV)
    ws = ws_for(S, 1, N)
    moe.moe_mx_product(S, K, 1, N, fmt, x.q, x.s, None, W.q, W.s, 2, y, ws)
    ok(ws)
    ref, mag = product_ref(x.v, W.v, [S])
    assert (np.abs(f64(y) - ref) <= K * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
def test_product_places_every_code_and_scale(fmt):
    """One weight and one activation are not zero: every (row, k) has to meet
    its own scale and its own place."""
    K, N, S = 1024, 264, 40
    rng = np.random.default_rng(3)
    for _ in range(6):
        xq, wq = np.zeros((S, K), np.int64), np.zeros((N, K), np.int64)
        k = rng.integers(0, K, S)
        one = 0x38 if fmt == mx.E4M3 else 2                       # the code of 1
        xq[np.arange(S), k] = one
        wq[:] = rng.integers(0, 16, (N, K))
        xs = rng.integers(117, 138, (S, K // 32))
        wsc = rng.integers(117, 138, (N, K // 32))
        y = torch.empty(S, N, device=DEV)
        ws = ws_for(S, 1, N)
        dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        moe.moe_mx_product(S, K, 1, N, fmt, dev(mx.pack(xq, fmt)), dev(mx.scale_rows(xs)), None,
                           dev(mx.pack(wq, mx.E2M1)), dev(mx.scale_rows(wsc)), 2, y, ws)
        ok(ws)
        want = mx.values(xq, xs, fmt) @ mx.values(wq, wsc, mx.E2M1).T
        assert np.array_equal(f64(y), want)                       # one product each: exact


def gated_ref(x, W1, W3, sizes, act):
    a, ma = product_ref(x, W1, sizes)
    b, mb = product_ref(x, W3, sizes)
    sig = 1 / (1 + np.exp(-a))
    g = sig if act else a * sig
    return a, b, g, ma, mb, g * b


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("sizes,d,f", [([1], 128, 128), ([2, 0, 1], 256, 384), ([37, 0, 128, 1, 200, 64], 640, 256),
                                       ([97, 95, 96], 512, 512), ([1] * 40, 256, 128), ([2, 1], 4096, 1408),
                                       ([1], 4096, 128), ([1] * 76, 2816, 128)])
def test_gated_matches_formula(fmt, act, sizes, d, f):
    rng = np.random.default_rng(len(sizes) + d + f)
    E, R = len(sizes), sum(sizes)
    S = R + 2
    x = mx.Matrix(rng, (S, d), fmt)
    x.s[R:] = 0xFF
    W1, W3 = mx.Matrix(rng, (E, f, d), mx.E2M1, 2 * d ** -0.5), mx.Matrix(rng, (E, f, d), mx.E2M1, d ** -0.5)
    h = torch.full((S, f), 7.0, dtype=torch.bfloat16, device=DEV)
    hq, hs = byte(S, f), byte(S, mx.pitch(f))
    ws = ws_for(S, E, f)
    args = (S, d, E, f, fmt, x.q, x.s, segments(sizes), W1.q, W1.s, W3.q, W3.s, act)
    moe.moe_mx_gated(*args, h, None, None, ws)
    ok(ws)
    moe.moe_mx_gated(*args, None, hq, hs, ws)
    ok(ws)
    assert (h[R:] == 7).all() and (hq[R:] == 0xA5).all() and (hs[R:] == 0xA5).all()
    a, b, g, ma, mb, ref = gated_ref(x.v, W1.v, W3.v, sizes, act)
    # errors of the two sums, through act (slope at most 1.1), and the fp32
    # activation: exp off by 2^-21 of itself and |a| 2^-24 of its argument's
    # rounding (|a| < 64 where h is not negligible), division and products.
    da, db = d * 2.0 ** -23 * ma, d * 2.0 ** -23 * mb
    tol = 1.1 * da * np.abs(b) + np.abs(g) * db + 1.1 * da * db + 2.0 ** -17 * np.abs(ref)
    got = f64(h[:R])
    assert (np.abs(got - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
    sc = hs[:R, :f // 32].cpu().numpy().astype(np.int64)
    pad = hs[:R, f // 32:]
    assert pad.numel() == 0 or int(pad.max()) == 0
    blocks, tb = np.abs(ref).reshape(R, -1, 32), tol.reshape(R, -1, 32)
    lo = mx.scale_code(np.maximum(blocks - tb, 0).max(axis=2), mx.E4M3)
    hi = mx.scale_code((blocks + tb).max(axis=2), mx.E4M3)
    assert ((sc >= lo) & (sc <= hi)).all()
    v = mx.values(hq[:R].cpu().numpy().astype(np.int64), sc, mx.E4M3)
    # half a step: 2^-4 relative, 2^-10 of the scale for subnormal codes
    half = np.maximum(2.0 ** -4 * (np.abs(ref) + tol), 2.0 ** -10 * np.repeat(mx.scale_value(sc), 32, axis=1))
    assert (np.abs(v - ref) <= tol + half).all()


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("sizes,d,f", [([700, 321, 1000], 2048, 4096), ([40, 61, 8, 77], 4096, 2048), ([3, 0, 9, 1], 4096, 4096)])
def test_products_give_the_same_bits_every_time(fmt, sizes, d, f):
    """Forty calls, other work between them: the pipelines hand over their
    buffers in time whatever the timing."""
    g = torch.Generator(device=DEV).manual_seed(7)
    E, S = len(sizes), sum(sizes)

    def codes(*shape, pitch):
        q = torch.randint(0, 255 if fmt == mx.E2M1 or len(shape) == 3 else 0x77, shape, generator=g, device=DEV, dtype=torch.uint8)
        return q, torch.randint(120, 130, (*shape[:-1], pitch), generator=g, device=DEV, dtype=torch.uint8)

    x, xs = codes(S, d if fmt == mx.E4M3 else d // 2, pitch=mx.pitch(d))
    W1, s1 = codes(E, f, d // 2, pitch=mx.pitch(d))
    W3, s3 = codes(E, f, d // 2, pitch=mx.pitch(d))
    off, ws = segments(sizes), ws_for(S, E, f)
    h, y = torch.empty(S, f, dtype=torch.bfloat16, device=DEV), torch.empty(S, f, device=DEV)
    first = None
    for i in range(40):
        moe.moe_mx_gated(S, d, E, f, fmt, x, xs, off, W1, s1, W3, s3, 1, h, None, None, ws)
        moe.moe_mx_product(S, d, E, f, fmt, x, xs, off, W3, s3, 2, y, ws)
        got = h.view(torch.int16).clone(), y.view(torch.int32).clone()
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), i
        if i % 3 == 0:
            torch.randn(1 << (16 + i % 8), device=DEV)
    ok(ws)


def test_products_pass_nan_scales_on():
    rng = np.random.default_rng(1)
    S, K, N = 9, 256, 136
    x, W = mx.Matrix(rng, (S, K), mx.E4M3), mx.Matrix(rng, (1, N, K), mx.E2M1)
    x.s[4, 3] = 255
    W.s[0, 7, 2] = 255
    y = torch.empty(S, N, device=DEV)
    ws = ws_for(S, 1, N)
    moe.moe_mx_product(S, K, 1, N, mx.E4M3, x.q, x.s, None, W.q, W.s, 2, y, ws)
    want = torch.zeros(S, N, dtype=torch.bool, device=DEV)
    want[4] = True
    want[:, 7] = True
    assert torch.equal(y.isnan(), want)
    h, hq, hs = torch.empty(S, 128, dtype=torch.bfloat16, device=DEV), byte(S, 128), byte(S, 16)
    V = mx.Matrix(rng, (1, 128, K), mx.E2M1)
    moe.moe_mx_gated(S, K, 1, 128, mx.E4M3, x.q, x.s, None, V.q, V.s, V.q, V.s, 0, h, None, None, ws)
    moe.moe_mx_gated(S, K, 1, 128, mx.E4M3, x.q, x.s, None, V.q, V.s, V.q, V.s, 0, None, hq, hs, ws)
    assert h[4].isnan().all() and not h[:4].isnan().any() and not h[5:].isnan().any()
    assert (hs[4, :4] == 255).all() and (hq[4] == 0).all() and (hs[5, :4] != 255).all()


@pytest.mark.parametrize("bad", [[0, 5, 4, 9], [-1, 2, 4, 9], [0, 2, 4, 12], [0, 11, 4, 9]])
def test_inconsistent_offsets_compute_nothing(bad):
    rng = np.random.default_rng(2)
    S, K, N = 9, 128, 128
    x, W = mx.Matrix(rng, (S, K), mx.E4M3), mx.Matrix(rng, (3, N, K), mx.E2M1)
    y = torch.full((S, N), 7.0, device=DEV)
    ws = ws_for(S, 3, N)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    moe.moe_mx_product(S, K, 3, N, mx.E4M3, x.q, x.s, off, W.q, W.s, 2, y, ws)
    assert moe.moe_get_device_error(ws) == (5, 8)
    assert (y == 7).all()
    h = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_gated(S, K, 3, N, mx.E4M3, x.q, x.s, off, W.q, W.s, W.q, W.s, 0, h, None, None, ws)
    assert moe.moe_get_device_error(ws) == (5, 8)
    assert (h == 7).all()
    # the next call on the workspace starts clean
    moe.moe_mx_product(S, K, 3, N, mx.E4M3, x.q, x.s, segments([3, 3, 3]), W.q, W.s, 2, y, ws)
    ok(ws)


def test_segments_may_start_behind_row_zero():
    rng = np.random.default_rng(5)
    S, K, N = 30, 256, 128
    x, W = mx.Matrix(rng, (S, K), mx.E4M3), mx.Matrix(rng, (2, N, K), mx.E2M1)
    y = torch.full((S, N), 7.0, device=DEV)
    ws = ws_for(S, 2, N)
    moe.moe_mx_product(S, K, 2, N, mx.E4M3, x.q, x.s, torch.tensor([4, 9, 21], dtype=torch.int32, device=DEV), W.q, W.s,
                       2, y, ws)
    ok(ws)
    ref, mag = product_ref(x.v[4:21], W.v, [5, 12])
    assert (np.abs(f64(y[4:21]) - ref) <= K * 2.0 ** -23 * mag).all()
    assert (y[:4] == 7).all() and (y[21:] == 7).all()


def test_empty_segments_write_nothing():
    rng = np.random.default_rng(4)
    S, K, N, E = 5, 256, 128, 4
    x, W = mx.Matrix(rng, (S, K), mx.E4M3), mx.Matrix(rng, (E, N, K), mx.E2M1)
    y, hq, hs = torch.full((S, N), 7.0, device=DEV), byte(S, N), byte(S, mx.pitch(N))
    ws = ws_for(S, E, N)
    for at in (0, 3, 5):
        off = torch.full((E + 1,), at, dtype=torch.int32, device=DEV)
        moe.moe_mx_product(S, K, E, N, mx.E4M3, x.q, x.s, off, W.q, W.s, 2, y, ws)
        moe.moe_mx_gated(S, K, E, N, mx.E4M3, x.q, x.s, off, W.q, W.s, W.q, W.s, 0, None, hq, hs, ws)
        ok(ws)
    assert (y == 7).all() and (hq == 0xA5).all() and (hs == 0xA5).all()


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
def test_many_experts_and_tile_borders(fmt):
    """256 experts, segments at and around the tile sizes, weights that start
    32 bytes into their allocation."""
    rng = np.random.default_rng(6)
    E, K, N = 256, 128, 16
    sizes = np.zeros(E, np.int64)
    sizes[[0, 3, 4, 77, 200, 254, 255]] = (192, 193, 1, 96, 97, 384, 16)
    S = int(sizes.sum())
    x, W = mx.Matrix(rng, (S, K), fmt), mx.Matrix(rng, (E, N, K), mx.E2M1)
    room = torch.empty(W.q.numel() + 64, dtype=torch.uint8, device=DEV)
    Wq = room[32:32 + W.q.numel()].view_as(W.q).copy_(W.q)
    y, ws = torch.empty(S, N, device=DEV), ws_for(S, E, N)
    moe.moe_mx_product(S, K, E, N, fmt, x.q, x.s, segments(sizes), Wq, W.s, 2, y, ws)
    ok(ws)
    ref, mag = product_ref(x.v, W.v, sizes)
    assert (np.abs(f64(y) - ref) <= K * 2.0 ** -23 * mag).all()


def test_indices_beyond_32_bits():
    """More than 2^31 elements in, and more than 2^31 out: the last rows."""
    rows, cols = 70000, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    q, s = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEV), torch.empty(rows, mx.pitch(cols), dtype=torch.uint8, device=DEV)
    moe.moe_mx_quantize(rows, cols, 0, x, cols, mx.E2M1, q, s)
    c, sc = mx.quantize(f64(x[-3:]), mx.E2M1)
    assert (q[-3:].cpu().numpy() == mx.pack(c, mx.E2M1)).all() and (s[-3:].cpu().numpy() == mx.scale_rows(sc)).all()
    T, d = rows * 2, cols // 2                                   # the same memory as rows of 16384
    h = x.view(T, d)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(h)
    moe.moe_rmsnorm(T, d, 0, h, d, 0, None, d, w, 1e-6, None, y, None, None)
    v = f64(h[-2:])
    n = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(1e-6)))
    assert (np.abs(f64(y[-2:]) - n) <= (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(n)).all()
    del x, h, y, q, s
    rng = np.random.default_rng(8)
    S, K, N = 33000, 128, 65536
    W = mx.Matrix(rng, (1, N, K), mx.E2M1)
    few = mx.Matrix(rng, (8, K), mx.E4M3)
    xq, xs = few.q.repeat(S // 8, 1), few.s.repeat(S // 8, 1)
    out, ws = torch.empty(S, N, dtype=torch.bfloat16, device=DEV), ws_for(S, 1, N)
    moe.moe_mx_product(S, K, 1, N, mx.E4M3, xq, xs, None, W.q, W.s, 0, out, ws)
    ok(ws)
    ref, mag = product_ref(few.v, W.v, [8])
    tol = K * 2.0 ** -23 * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(f64(out[-8:]) - ref) <= tol).all()
    assert torch.equal(out[:8], out[-8:])


# ------------------------------------------------------------ used together

def layer(rng, T, d, E, f, k):
    g = torch.Generator(device=DEV).manual_seed(T)
    p = dict(h=torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16),
             delta=torch.randn(T, d, generator=g, device=DEV),
             w=(1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16),
             Wg=(torch.randn(E, d, generator=g, device=DEV) * d ** -0.5).to(torch.bfloat16))
    p.update(W1=mx.Matrix(rng, (E, f, d), mx.E2M1, d ** -0.5), W3=mx.Matrix(rng, (E, f, d), mx.E2M1, d ** -0.5),
             W2=mx.Matrix(rng, (E, d, f), mx.E2M1, f ** -0.5))
    return p


def forward(p, T, d, E, f, k, out, ws, h_out=None, delta=True, stream=None, bias=None):
    moe.moe_forward_mx(T, d, E, f, k, p["h"], p["delta"] if delta else None, p["w"], 1e-6, h_out, p["Wg"], bias, p["W1"].q,
                       p["W1"].s, p["W3"].q, p["W3"].s, p["W2"].q, p["W2"].s, out, ws, stream=stream)


def composed(p, T, d, E, f, k, delta=True):
    """The layer from the separate entry points; also its routing."""
    S = T * k
    ho, x = torch.empty_like(p["h"]), torch.empty_like(p["h"])
    q, s = byte(T, d), byte(T, mx.pitch(d))
    moe.moe_rmsnorm(T, d, 0, p["h"], d, 2, p["delta"] if delta else None, d, p["w"], 1e-6, ho, x, q, s)
    ws = byte(moe.moe_workspace_size(T, d, E, f, k))
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    off, row = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    moe.moe_route(T, d, E, k, x, p["Wg"], None, idx, w, None, ws)
    xp = torch.empty(S, d, dtype=torch.bfloat16, device=DEV)
    moe.moe_permute(T, d, E, k, x, idx, off, row, xp, ws)
    token = torch.empty(S, dtype=torch.long, device=DEV)
    token[row.long().flatten()] = torch.arange(T, device=DEV).repeat_interleave(k)
    hq, hs = byte(S, f), byte(S, mx.pitch(f))
    mws = ws_for(S, E, max(f, d))
    moe.moe_mx_gated(S, d, E, f, mx.E4M3, q[token].contiguous(), s[token].contiguous(), off, p["W1"].q, p["W1"].s,
                     p["W3"].q, p["W3"].s, 0, None, hq, hs, mws)
    ok(mws)
    y = torch.empty(S, d, dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_product(S, f, E, d, mx.E4M3, hq, hs, off, p["W2"].q, p["W2"].s, 0, y, mws)
    ok(mws)
    out = torch.empty(T, d, device=DEV)
    moe.moe_combine(T, d, k, y.float(), row, w, None, out)
    return out, ho, q, s, idx, w


LAYERS = [(1, 256, 8, 512, 2), (5, 128, 4, 128, 1), (64, 512, 32, 256, 4), (300, 1152, 8, 640, 2), (129, 256, 60, 128, 8)]


@pytest.mark.parametrize("T,d,E,f,k", LAYERS)
@pytest.mark.parametrize("delta", [True, False])
def test_forward_is_the_composition_and_the_formula(T, d, E, f, k, delta):
    rng = np.random.default_rng(T)
    p = layer(rng, T, d, E, f, k)
    out = torch.empty(T, d, device=DEV)
    ho = torch.empty_like(p["h"])
    ws = byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k), fill=0xFF)
    forward(p, T, d, E, f, k, out, ws, ho, delta)
    ok(ws)
    want, ho2, q, s, idx, w = composed(p, T, d, E, f, k, delta)
    assert torch.equal(ho, ho2)
    # the same kernels on the same rows; moe_combine's own order of the k sums
    assert torch.allclose(out, want, rtol=0, atol=float(want.abs().max()) * k * 2.0 ** -23)
    # the layer in 64 bits from the quantised rows and the routing
    xv = mx.values(q.cpu().numpy().astype(np.int64), s[:, :d // 32].cpu().numpy().astype(np.int64), mx.E4M3)
    ref, tol = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e, wt = int(idx[t, j]), float(w[t, j])
            a, b = p["W1"].v[e] @ xv[t], p["W3"].v[e] @ xv[t]
            h = a / (1 + np.exp(-a)) * b
            c, sc = mx.quantize(h[None], mx.E4M3)
            hv = mx.values(c, sc, mx.E4M3)[0]
            y = p["W2"].v[e] @ hv
            ref[t] += wt * y
            # bf16 rows; of the codes of h, at most those near a border differ,
            # by a step (2^-3): taken as 1 in 1000, of random sign
            tol[t] += wt * (2.0 ** -8 * np.abs(y) + 2.0 ** -3 * np.sqrt((p["W2"].v[e] ** 2 @ hv ** 2) * 1e-3)
                            + (d + f) * 2.0 ** -23 * (np.abs(p["W2"].v[e]) @ np.abs(hv)))
    assert (np.abs(f64(out) - ref) <= tol * 4 + 1e-12).all()


def test_forward_with_a_bias_and_in_place():
    """A router bias that sends every token to experts 1 and 6, and the
    residual stream updated where it stands."""
    T, d, E, f, k = 70, 256, 8, 256, 2
    p = layer(np.random.default_rng(2), T, d, E, f, k)
    bias = torch.full((E,), -1e4, device=DEV)
    bias[[1, 6]] = 1e4
    out, ws = torch.empty(T, d, device=DEV), byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k))
    want = (p["h"].float() + p["delta"]).to(torch.bfloat16)
    stored = p["h"].clone()
    forward(p, T, d, E, f, k, out, ws, bias=bias)
    assert torch.equal(p["h"], stored)
    first = out.clone()
    forward(p, T, d, E, f, k, out, ws, p["h"], bias=bias)
    ok(ws)
    assert torch.equal(p["h"], want) and torch.equal(out, first)
    # the norm's bf16 rows through the two experts, in 64 bits from its 8-bit rows
    ho, y, q, s = torch.empty_like(want), torch.empty_like(want), byte(T, d), byte(T, mx.pitch(d))
    moe.moe_rmsnorm(T, d, 0, want, d, 0, None, d, p["w"], 1e-6, ho, y, q, s)
    xv = mx.values(q.cpu().numpy().astype(np.int64), s[:, :d // 32].cpu().numpy().astype(np.int64), mx.E4M3)
    a = f64(y) @ f64(p["Wg"]).T + f64(bias)
    e = np.exp(a[:, [1, 6]] - a[:, [1, 6]].max(axis=1, keepdims=True))
    wt = e / e.sum(axis=1, keepdims=True)
    ref = np.zeros((T, d))
    for i, j in enumerate((1, 6)):
        g, b = xv @ p["W1"].v[j].T, xv @ p["W3"].v[j].T
        c, sc = mx.quantize(g / (1 + np.exp(-g)) * b, mx.E4M3)
        ref += wt[:, i:i + 1] * (mx.values(c, sc, mx.E4M3) @ p["W2"].v[j].T)
    # logits near 1e4 are known to 2^-24 * 1e4 * a few (the weights to that),
    # rows are rounded to bf16, few codes of h differ by a step
    assert np.abs(f64(out) - ref).max() <= 2.0 ** -6 * np.abs(ref).max()


def test_forward_in_graphs_and_on_streams():
    """Two graphs of two layers on workspaces of their own, replayed in turn
    and together with an eager call on another stream."""
    T, d, E, f, k = 33, 512, 8, 384, 2
    rng = np.random.default_rng(9)
    ps = [layer(rng, T, d, E, f, k), layer(rng, T, d, E, f, k)]
    wants = []
    for p in ps:
        out, ws = torch.empty(T, d, device=DEV), byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k))
        forward(p, T, d, E, f, k, out, ws)
        wants.append(out)
    graphs, outs, wss = [], [], []
    for p in ps:
        out, ws = torch.zeros(T, d, device=DEV), byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p["h"].add_(0)                       # a kernel of another library before the first node
            forward(p, T, d, E, f, k, out, ws)
        graphs.append(g), outs.append(out), wss.append(ws)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(side)
        for o, w in zip(outs, wants):
            assert torch.equal(o, w)
    for ws in wss:
        ok(ws)
    out = torch.zeros(T, d, device=DEV)
    ws = byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k))
    side.wait_stream(torch.cuda.current_stream())
    forward(ps[0], T, d, E, f, k, out, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, wants[0])


def test_every_operator_in_one_graph_after_a_memset():
    """The single-kernel operators captured right behind a memset and a copy,
    replayed on new inputs."""
    T, d = 37, 544
    x, y, z = torch.zeros(T, d, device=DEV), torch.empty(T, d, device=DEV), torch.zeros(T, d, device=DEV)
    w = torch.ones(d, device=DEV)
    q, s = byte(T, d), byte(T, mx.pitch(d))
    src = torch.zeros(T, d, device=DEV)
    q4, s4 = byte(T, d // 2), byte(T, mx.pitch(d))

    def run():
        z.zero_()
        x.copy_(src)
        moe.moe_rmsnorm(T, d, 2, x, d, 2, z, d, w, 1e-6, None, y, q, s)
        moe.moe_mx_quantize(T, d, 2, y, d, mx.E2M1, q4, s4)

    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in range(3):
        src.copy_(torch.randn(T, d, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
        g.replay()
        v = f64(src)
        n = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(1e-6)))
        assert (np.abs(f64(y) - n) <= 5 * 2.0 ** -24 * np.abs(n)).all()
        c, sc = mx.quantize(f64(y), mx.E2M1)
        assert (q4.cpu().numpy() == mx.pack(c, mx.E2M1)).all() and (s4.cpu().numpy() == mx.scale_rows(sc)).all()


def test_the_examples_of_the_readme_run():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "moe." in b]
    assert len(blocks) == 2
    names = {}
    exec("\n".join(blocks), names)
    torch.cuda.synchronize()
    assert names["out"].isfinite().all() and names["stream"].isfinite().all()
    assert moe.moe_get_device_error(names["ws"])[0] == 0


# ------------------------------------------- sums that meet in the workspace
# Units that do not fill the last turn of the CTA pairs are cut along K where
# that saves more than it costs, by the number of units, the chunks of 512 in
# K and the rows of the call.  A workspace holds, behind the header of 256
# bytes, one counter for every cut unit, CTA and epilogue warp (80 x 2 x 8),
# which says how many of the unit's parts have come in.

COUNTERS = 80 * 2 * 8 * 4


def cut_units(ws, at=256):
    """How many units the last call on the workspace cut (a call that can cut
    none leaves the counters alone)."""
    c = ws[at:at + COUNTERS].view(torch.int32).view(80, 16)
    return int((c > 0).any(dim=1).sum())


def units(sizes, N, rows_blk, S):
    """Units of a launch: tiles of at most 96 or 192 rows times blocks of N."""
    most = 96 if -(-S // len(sizes)) <= 64 else 192
    return sum(-(-n // most) for n in sizes) * -(-N // rows_blk)


class Codes:
    """Random 4-bit weights [E, rows, cols] of about the size cols^-1/2, made
    on the GPU: `q`, `s` as the library takes them, `v` their fp64 values."""

    def __init__(self, g, E, rows, cols):
        self.q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
        self.s = torch.zeros(E, rows, mx.pitch(cols), dtype=torch.uint8, device=DEV)
        self.s[..., :cols // 32] = 127 - round(np.log2(3 * cols ** 0.5)) + \
            torch.randint(0, 2, (E, rows, cols // 32), generator=g, device=DEV, dtype=torch.uint8)
        self.cols = cols

    def matrix(self, e):
        v = torch.from_numpy(np.concatenate([mx.grid(mx.E2M1), -mx.grid(mx.E2M1)])).to(DEV)
        c = torch.stack([self.q[e] & 15, self.q[e] >> 4], dim=-1).flatten(-2).long()
        s = torch.exp2(self.s[e, :, :self.cols // 32].double() - 127)
        return v[c] * s.repeat_interleave(32, dim=-1)


def codes_ref(x, W, sizes):
    """(y, sum of magnitudes) in 64 bits, on the GPU, of fp64 rows and Codes."""
    y, a, r = [], [], 0
    for e, n in enumerate(sizes):
        if n:
            m, rows = W.matrix(e), torch.from_numpy(x[r:r + n]).to(DEV)
            y.append(rows @ m.T), a.append(rows.abs() @ m.abs().T)
        r += n
    return torch.cat(y).cpu().numpy(), torch.cat(a).cpu().numpy()


CUT = [
    ([40], 8192, 512), ([33, 0, 40], 10240, 264), ([100, 5], 16384, 136),   # tiles of at most 96 rows
    ([80], 8192, 264), ([190], 16384, 24), ([200, 100], 16384, 264),        # of at most 192 rows
    ([1] * 5, 4096, 4096), ([9, 0, 30, 17, 3, 1], 8192, 4096),   # six of 80 units cut, the others whole
]


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("sizes,K,N", CUT)
@pytest.mark.parametrize("yt", [0, 2])
@pytest.mark.parametrize("behind", [0, 2])
def test_product_of_cut_units_matches_formula(fmt, sizes, K, N, yt, behind):
    rng = np.random.default_rng(len(sizes) + K + N)
    E, R = len(sizes), sum(sizes)
    S = R + behind                                 # rows behind the last segment
    x = mx.Matrix(rng, (S, K), fmt)
    x.s[R:] = 0xFF
    W = Codes(torch.Generator(device=DEV).manual_seed(K + N), E, N, K)
    t = mx.TORCH[yt]
    y = torch.full((S, N), 7.0, dtype=t, device=DEV)
    ws = ws_for(S, E, N)
    args = (S, K, E, N, fmt, x.q, x.s, segments(sizes), W.q, W.s, yt)
    moe.moe_mx_product(*args, y, ws)
    ok(ws)
    n = cut_units(ws)
    assert 0 < n <= units(sizes, N, 256, S)
    if units(sizes, N, 256, S) >= 80:
        assert n < units(sizes, N, 256, S)
    assert (y[R:] == 7).all()
    ref, mag = codes_ref(x.v[:R], W, sizes)
    err = np.abs(f64(y[:R]) - ref)
    assert (err <= K * 2.0 ** -23 * mag * (1 + HALF[t]) + HALF[t] * np.abs(ref)).all()
    for _ in range(3):                             # the same workspace again: the same bits
        y2 = torch.full((S, N), 7.0, dtype=t, device=DEV)
        moe.moe_mx_product(*args, y2, ws)
        assert torch.equal(y, y2)
    ok(ws)


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("sizes,K,N", [([40], 8192, 512), ([150], 16384, 264), ([9, 0, 30, 17, 3, 1], 8192, 4096)])
def test_cut_units_lose_no_product(fmt, sizes, K, N):
    """Whole numbers: every sum is one below 2^24, so the result is exact
    whatever the order, and a chunk left out or counted twice shows."""
    rng = np.random.default_rng(K + N)
    E, S = len(sizes), sum(sizes)
    one = 0x38 if fmt == mx.E4M3 else 2                           # the code of 1
    xq = one * rng.integers(0, 2, (S, K))
    x = torch.from_numpy((xq > 0).astype(np.float64)).to(DEV)
    W = Codes(torch.Generator(device=DEV).manual_seed(K + N), E, N, K)
    W.q &= 0xAA                                                   # 0, 1, -0, -1
    W.s[..., :K // 32] = 127
    xs = torch.from_numpy(mx.scale_rows(np.full((S, K // 32), 127))).to(DEV)
    y, ws = torch.empty(S, N, device=DEV), ws_for(S, E, N)
    moe.moe_mx_product(S, K, E, N, fmt, torch.from_numpy(mx.pack(xq, fmt)).to(DEV), xs, segments(sizes), W.q, W.s, 2, y, ws)
    ok(ws)
    assert cut_units(ws) > 0
    r = 0
    for e, n in enumerate(sizes):
        assert torch.equal(y[r:r + n].double(), x[r:r + n] @ W.matrix(e).T), e
        r += n


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("sizes,d,f", [([40], 8192, 128), ([100], 16384, 256), ([190], 16384, 128), ([150, 60], 16384, 128),
                                       ([1] * 5, 4096, 2048), ([9, 0, 30, 17, 3, 1], 8192, 2048)])
def test_gated_of_cut_units_matches_formula(fmt, act, sizes, d, f):
    rng = np.random.default_rng(len(sizes) + d + f)
    E, R = len(sizes), sum(sizes)
    S = R + 2
    x = mx.Matrix(rng, (S, d), fmt)
    x.s[R:] = 0xFF
    g = torch.Generator(device=DEV).manual_seed(d + f)
    W1, W3 = Codes(g, E, f, d), Codes(g, E, f, d)
    h = torch.full((S, f), 7.0, dtype=torch.bfloat16, device=DEV)
    hq, hs = byte(S, f), byte(S, mx.pitch(f))
    ws = ws_for(S, E, f)
    args = (S, d, E, f, fmt, x.q, x.s, segments(sizes), W1.q, W1.s, W3.q, W3.s, act)
    n = units(sizes, f, 128, S)
    moe.moe_mx_gated(*args, h, None, None, ws)
    ok(ws)
    assert 0 < cut_units(ws) <= n and (n < 80 or cut_units(ws) < n)
    moe.moe_mx_gated(*args, None, hq, hs, ws)
    ok(ws)
    assert 0 < cut_units(ws)
    assert (h[R:] == 7).all() and (hq[R:] == 0xA5).all() and (hs[R:] == 0xA5).all()
    # as in test_gated_matches_formula
    (a, ma), (b, mb) = codes_ref(x.v[:R], W1, sizes), codes_ref(x.v[:R], W3, sizes)
    g = 1 / (1 + np.exp(-a)) * (1 if act else a)
    ref = g * b
    da, db = d * 2.0 ** -23 * ma, d * 2.0 ** -23 * mb
    tol = 1.1 * da * np.abs(b) + np.abs(g) * db + 1.1 * da * db + 2.0 ** -17 * np.abs(ref)
    assert (np.abs(f64(h[:R]) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
    sc = hs[:R, :f // 32].cpu().numpy().astype(np.int64)
    blocks, tb = np.abs(ref).reshape(R, -1, 32), tol.reshape(R, -1, 32)
    lo = mx.scale_code(np.maximum(blocks - tb, 0).max(axis=2), mx.E4M3)
    hi = mx.scale_code((blocks + tb).max(axis=2), mx.E4M3)
    assert ((sc >= lo) & (sc <= hi)).all()
    v = mx.values(hq[:R].cpu().numpy().astype(np.int64), sc, mx.E4M3)
    half = np.maximum(2.0 ** -4 * (np.abs(ref) + tol), 2.0 ** -10 * np.repeat(mx.scale_value(sc), 32, axis=1))
    assert (np.abs(v - ref) <= tol + half).all()
    for _ in range(3):
        h2, q2, s2 = torch.full_like(h, 7.0), byte(S, f), byte(S, mx.pitch(f))
        moe.moe_mx_gated(*args, h2, None, None, ws)
        moe.moe_mx_gated(*args, None, q2, s2, ws)
        assert torch.equal(h, h2) and torch.equal(hq, q2) and torch.equal(hs, s2)
    ok(ws)


# rows, widths and experts of which both products cut units: all of them (6144
# -> 4096, one expert hit), and two of 150 in the up projections (4096 -> 9600)
@pytest.mark.parametrize("T,d,E,f,k", [(1, 6144, 2, 4096, 1), (1, 4096, 2, 9600, 2), (3, 4096, 2, 9600, 2)])
def test_forward_of_cut_units(T, d, E, f, k):
    """The layer's own counters and scratch: a workspace filled with ones, the
    same one again on other inputs, and replayed from a graph."""
    g = torch.Generator(device=DEV).manual_seed(T + d)
    S = T * k
    p = dict(h=None, delta=None, w=(1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16),
             Wg=(torch.randn(E, d, generator=g, device=DEV) * d ** -0.5).to(torch.bfloat16),
             W1=Codes(g, E, f, d), W3=Codes(g, E, f, d), W2=Codes(g, E, d, f))
    inputs = [(torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16), torch.randn(T, d, generator=g, device=DEV))
              for _ in range(3)]
    ws = byte(moe.moe_forward_mx_workspace_size(T, d, E, f, k), fill=0xFF)
    outs = []
    for h, delta in inputs + inputs[:1]:
        p.update(h=h, delta=delta)
        out = torch.full((T, d), float("nan"), device=DEV)
        forward(p, T, d, E, f, k, out, ws)
        ok(ws)
        # behind the header and the router's tile counter
        assert cut_units(ws, 512) > 0 and cut_units(ws, 512 + COUNTERS) > 0
        outs.append(out)
    assert torch.equal(outs[0], outs[3])
    src_h, src_delta = torch.empty_like(inputs[0][0]), torch.empty_like(inputs[0][1])
    p.update(h=src_h, delta=src_delta)
    out = torch.empty(T, d, device=DEV)
    src_h.copy_(inputs[0][0]), src_delta.copy_(inputs[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(p, T, d, E, f, k, out, ws)
    for (h, delta), want in list(zip(inputs, outs)) * 2:
        src_h.copy_(h), src_delta.copy_(delta)
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, want)
    ok(ws)
    # the separate calls, and the formula in 64 bits from their rows and routing
    for (h, delta), out in zip(inputs[:2], outs):
        p.update(h=h, delta=delta)
        want, _, q, s, idx, w = composed(p, T, d, E, f, k)
        assert torch.allclose(out, want, rtol=0, atol=float(want.abs().max()) * k * 2.0 ** -23)
        xv = torch.from_numpy(mx.values(q.cpu().numpy().astype(np.int64), s[:, :d // 32].cpu().numpy().astype(np.int64), mx.E4M3)).to(DEV)
        ref, tol = torch.zeros(T, d, dtype=torch.float64, device=DEV), torch.zeros(T, d, dtype=torch.float64, device=DEV)
        for t in range(T):
            for j in range(k):
                e, wt = int(idx[t, j]), float(w[t, j])
                a, b = p["W1"].matrix(e) @ xv[t], p["W3"].matrix(e) @ xv[t]
                hh = a * torch.sigmoid(a) * b
                c, sc = mx.quantize(f64(hh)[None], mx.E4M3)
                hv = torch.from_numpy(mx.values(c, sc, mx.E4M3)[0]).to(DEV)
                W2 = p["W2"].matrix(e)
                y = W2 @ hv
                ref[t] += wt * y
                # as in test_forward_is_the_composition_and_the_formula
                tol[t] += wt * (2.0 ** -8 * y.abs() + 2.0 ** -3 * torch.sqrt((W2 ** 2 @ hv ** 2) * 1e-3)
                                + (d + f) * 2.0 ** -23 * (W2.abs() @ hv.abs()))
        assert ((out.double() - ref).abs() <= tol * 4 + 1e-12).all()
