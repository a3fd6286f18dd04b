"""The experts' gate act(g) * b at values whose product or exponential leaves
fp32's range, in every kernel that computes it.

Every case makes g and b of hidden column f exactly: x has a one in its first
column and zeros elsewhere, the first columns of W1 and W3 hold g and b, and
W2 is the identity, so that output column f is h[f] as the kernel stores it.
"""
import numpy as np
import pytest
import torch

import mx_util as mx
import sparse_mixture_experts_histogram_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (g, b), all of them bf16 values
PLAIN = [(3.0, -5.0), (-3.0, 5.0), (0.5, 0.25), (-20.0, 7.0), (0.0, 9.0), (4.0, 0.0), (64.0, 2.0), (-86.5, 2.0 ** 100)]
# g far below zero: act(g) is next to nothing, whatever g * b or exp(-g) is
SMALL = [(-2.0 ** 66, 2.0 ** 66), (-2.0 ** 66, -2.0 ** 66), (-2.0 ** 100, 2.0 ** 120), (-2.0 ** 126, -2.0 ** 126),
         (-96.0, 2.0 ** 126), (-88.0, 2.0 ** 120), (-88.0, -1.0), (-100.0, 1.5 * 2.0 ** 126), (-87.5, 2.0 ** 125),
         (-128.0, 2.0 ** 126), (-192.0, 2.0 ** 126)]
# g * b leaves the range, act(g) * b does not
LARGE = [(-50.0, 2.0 ** 126), (1.75, 1.3125 * 2.0 ** 127), (-20.0, -2.0 ** 126), (-6.0, 2.0 ** 126)]


def gate(g, b, act):
    """act(g) * b in 64 bits and how far fp32 may be off: exp(-|g|) by the
    rounding of its argument, |g| log2(e) below 256 in fp32 (half a step, 2^-17,
    and the constant's 2^-25 of 256: together ln 2 (2^-17 + 2^-17) = 2^-16.5 of
    the value; a larger |g| leaves nothing), the division and products by a few
    2^-23; below the smallest normal by 2^-149."""
    g, b = np.asarray(g, np.float64), np.asarray(b, np.float64)
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-g))
    ref = (sig if act else g * sig) * b
    return ref, 2.0 ** -16 * np.abs(ref) + 2.0 ** -149


def columns(pairs, n, rng):
    """n columns with every pair, the rest repeats, in random order."""
    p = np.array([pairs[i % len(pairs)] for i in range(n)])
    return p[rng.permutation(n)]


def check(y, gb, act, half, tiny):
    ref, tol = gate(gb[:, 0], gb[:, 1], act)
    y = y.double().cpu().numpy()
    assert (np.abs(y - ref) <= tol + half * (np.abs(ref) + tol) + tiny).all(), \
        [(tuple(gb[f]), y[r, f], ref[f]) for r, f in np.argwhere(~(np.abs(y - ref) <= tol + half * (np.abs(ref) + tol) + tiny))[:8]]


def first_column(v, d):
    W = torch.zeros(1, len(v), d, dtype=torch.bfloat16, device=DEV)
    W[0, :, 0] = torch.from_numpy(np.asarray(v)).to(DEV)
    return W


@pytest.mark.parametrize("S", [1, 3, 40, 100, 300])
@pytest.mark.parametrize("d", [128, 1152])
def test_expert_ffn_gate(S, d):
    gb = columns(PLAIN + SMALL + LARGE, d, np.random.default_rng(S))
    W1, W3 = first_column(gb[:, 0], d), first_column(gb[:, 1], d)
    W2 = torch.eye(d, dtype=torch.bfloat16, device=DEV)[None].contiguous()
    x = torch.zeros(S, d, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    off = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    y, ws = torch.empty(S, d, device=DEV), torch.empty(moe.moe_workspace_size(S, d, 1, d, 1), dtype=torch.uint8, device=DEV)
    moe.moe_expert_ffn(S, d, 1, d, x, off, W1, W3, W2, y, ws)
    assert moe.moe_get_device_error(ws)[0] == 0
    check(y, gb, 0, 2.0 ** -8, 2.0 ** -134)


@pytest.mark.parametrize("T,d", [(5, 128), (200, 256), (5, 1152)])
@pytest.mark.parametrize("act", [0, 1])
def test_forward_gate(T, d, act):
    """d <= 1024: the narrow-layer kernel."""
    gb = columns(PLAIN + SMALL + LARGE[:1 if act else None], d, np.random.default_rng(T))
    W1, W3 = first_column(gb[:, 0], d), first_column(gb[:, 1], d)
    W2 = torch.eye(d, dtype=torch.bfloat16, device=DEV)[None].contiguous()
    Wg = torch.zeros(1, d, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    out = torch.empty(T, d, device=DEV)
    ws = torch.empty(moe.moe_workspace_size(T, d, 1, d, 1), dtype=torch.uint8, device=DEV)
    v = moe.MoEVariant(weights=moe.WEIGHTS_SOFTMAX_TOPK, activation=act, capacity_factor=0.0)
    moe.moe_forward_variant(T, d, 1, d, 1, x, Wg, None, W1, W3, W2, 0, None, None, None, v, out, ws)
    assert moe.moe_get_device_error(ws)[0] == 0
    check(out, gb, act, 2.0 ** -8, 2.0 ** -134)


@pytest.mark.parametrize("T", [1, 5, 100, 300])
def test_forward_fp8_gate(T):
    """g and b from the rows' scales; h is kept within fp16's range."""
    d = 256
    pairs = [p for p in PLAIN + SMALL + LARGE if abs(gate(*p, 0)[0]) < 6e4]
    gb = columns(pairs, d, np.random.default_rng(T))

    def stored(v):
        q = torch.zeros(1, d, d, dtype=torch.uint8)
        q[0, :, 0] = torch.from_numpy(np.where(np.signbit(v), 0xB8, 0x38).astype(np.uint8))    # -1 and 1
        return q.to(DEV), torch.from_numpy(np.abs(v).astype(np.float32))[None].to(DEV)

    (q1, s1), (q3, s3) = stored(gb[:, 0]), stored(gb[:, 1])
    q2 = (torch.eye(d, dtype=torch.uint8) * 0x38)[None].contiguous().to(DEV)
    s2 = torch.ones(1, d, device=DEV)
    Wg = torch.zeros(1, d, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    out, ws = torch.empty(T, d, device=DEV), torch.empty(moe.moe_workspace_size(T, d, 1, d, 1), dtype=torch.uint8, device=DEV)
    moe.moe_forward_fp8(T, d, 1, d, 1, x, Wg, None, q1, s1, q3, s3, q2, s2, out, ws)
    assert moe.moe_get_device_error(ws)[0] == 0
    check(out, gb, 0, 2.0 ** -11, 2.0 ** -25)


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("S,d", [(1, 128), (70, 128), (300, 256), (3, 4096)])
def test_mx_gated_gate(fmt, act, S, d):
    """One non-zero product a sum: x is 1.375 or 1, 1.5 in 4 bits, W a power of
    two times 1 or 1.5 (E2M1 codes with scales up to 2^127).  (3, 4096): the
    sums meet in the workspace."""
    f = 256
    rng = np.random.default_rng(S)
    x0 = np.where(np.arange(S) % 2, 1.0, 1.5 if fmt == mx.E2M1 else 1.375)
    pairs = [(-2.0 ** 66, 2.0 ** 66), (-2.0 ** 66, -1.5 * 2.0 ** 66), (-2.0 ** 100, 2.0 ** 120), (-96.0, 2.0 ** 126),
             (-64.0, 2.0 ** 120), (-64.0, -1.0), (-128.0, 2.0 ** 126), (-48.0, 2.0 ** 125), (3.0, -4.0), (-3.0, 4.0),
             (0.5, 1.5), (-16.0, 6.0), (64.0, 2.0), (-2.0 ** 126, -2.0 ** 126), (0.0, 3.0), (1.0, 0.0)]
    if not act:
        pairs += [(1.0, 2.0 ** 127), (-12.0, 2.0 ** 126)]
    # a block of 32 columns holds results of one size
    ref = [abs(gate(g, b, act)[0]) for g, b in pairs]
    order = [pairs[i] for i in np.argsort(ref)]
    gb = np.array([order[i * len(order) // f] for i in range(f)])

    def stored(v):
        """Rows whose first value is v = c 2^e, c in (0, 1, 1.5), and whose others are 0."""
        m, e = np.frexp(np.abs(v))
        c = np.zeros((f, d), np.int64)
        sc = np.full((f, d // 32), 127)
        c[:, 0] = np.where(v == 0, 0, np.where(m == 0.75, 3, 2)) + 8 * np.signbit(v)
        sc[:, 0] = np.where(v == 0, 127, e - 1 + 127)
        assert np.array_equal(mx.values(c, sc, mx.E2M1)[:, 0], v)
        return (torch.from_numpy(mx.pack(c, mx.E2M1))[None].contiguous().to(DEV),
                torch.from_numpy(mx.scale_rows(sc))[None].contiguous().to(DEV))

    (q1, s1), (q3, s3) = stored(gb[:, 0]), stored(gb[:, 1])
    xc = np.zeros((S, d), np.int64)
    xc[:, 0] = np.where(x0 == 1, 0x38, 0x3B) if fmt == mx.E4M3 else np.where(x0 == 1, 2, 3)
    xsc = np.full((S, d // 32), 127)
    assert np.array_equal(mx.values(xc, xsc, fmt)[:, 0], x0)
    xq, xs = torch.from_numpy(mx.pack(xc, fmt)).to(DEV), torch.from_numpy(mx.scale_rows(xsc)).to(DEV)
    ws = torch.full((moe.moe_mx_workspace_size(S, 1, f),), 0xFF, dtype=torch.uint8, device=DEV)
    h = torch.empty(S, f, dtype=torch.bfloat16, device=DEV)
    hq, hs = torch.empty(S, f, dtype=torch.uint8, device=DEV), torch.empty(S, mx.pitch(f), dtype=torch.uint8, device=DEV)
    args = (S, d, 1, f, fmt, xq, xs, None, q1, s1, q3, s3, act)
    moe.moe_mx_gated(*args, h, None, None, ws)
    assert moe.moe_get_device_error(ws)[0] == 0
    moe.moe_mx_gated(*args, None, hq, hs, ws)
    assert moe.moe_get_device_error(ws)[0] == 0
    want, tol = gate(x0[:, None] * gb[:, 0], x0[:, None] * gb[:, 1], act)
    assert (np.abs(want) < 3.38e38).all()
    got = h.double().cpu().numpy()
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134).all()
    sc = hs[:, :f // 32].cpu().numpy().astype(np.int64)
    assert (sc < 255).all()
    v = mx.values(hq.cpu().numpy().astype(np.int64), sc, mx.E4M3)
    # half a step: 2^-4 relative, 2^-10 of the scale for subnormal codes
    half = np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * np.repeat(mx.scale_value(sc), 32, axis=1))
    assert (np.abs(v - want) <= tol + half).all()
