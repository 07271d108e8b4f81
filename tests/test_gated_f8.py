"""The gated unit silu(g) u of the F8 products by itself, over the whole range of g.

Every gate and up value is put together exactly: rows of x have a 1 at the first column of each
group, a gate row has three digits of four bits there in groups 0 to 2 (scales 2^0, 2^-4, 2^-8),
an up row one digit in group 3, and the scales of x move gate and up over the range of
exponents.  So the product has no error, which the plain float32 product shows, and only the
unit's is left: 17 * 2^-24 of the result (an exponential within 2^-22 squared and nine
roundings), 2^-240 of u where its factor is below the normal numbers, and the step of a
subnormal result."""

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gpu_util import require_gpu, to_dev, to_host
from oracle import f8

pytestmark = pytest.mark.gpu

GATE = [-126, -20, -3, 0, 2, 3, 4, 5, 6, 7, 12, 60, 126]   # exponents of the gates' magnitudes
UP = [-20, 0, 100]


def _case(n, seed):
    """(weights, x, g, u): n hidden columns, a row for every pair of exponents."""
    rng = np.random.default_rng(seed)
    K, N = 512, 2 * n
    values = np.zeros((N, K))
    sign = rng.choice([-1.0, 1.0], (n, 1))
    digits = 1 + rng.integers(0, 8, (n, 3)) / 8
    values[0::2, [0, 128, 256]] = sign * digits
    up = rng.choice([-1.0, 1.0], n) * (1 + rng.integers(0, 8, n) / 8)
    values[1::2, 384] = up
    wc = f8.e4m3_encode(values)
    ws = np.tile(np.array([127, 123, 119, 127], np.uint8), (-(-N // 128), 1))
    pairs = [(a, b) for a in GATE for b in UP]
    xc = np.zeros((len(pairs), K), np.uint8)
    xc[:, ::128] = f8.e4m3_encode(np.ones(1))[0]
    xs = np.array([[127 + a] * 3 + [127 + b] for a, b in pairs], np.uint8)
    a, b = (np.exp2(np.array(e, np.float64))[:, None] for e in zip(*pairs))
    g = a * (sign * digits * [1, 2.0 ** -4, 2.0 ** -8]).sum(1)
    return (wc, ws), (xc, xs), g, b * up


def _run(w, x, n, repeat, experts, act, dtype):
    """The case's rows `repeat` times over, as a dense product or as three experts."""
    (wc, ws), (xc, xs) = w, x
    M = repeat * xc.shape[0]
    xc, xs = (to_dev(np.tile(a, (repeat, 1))) for a in (xc, xs))
    Y = torch.empty((M, n if act == "swiglu" else 2 * n), device="cuda", dtype=dtype)
    if experts:
        off = np.array([0, M // 3, M // 3, M], np.int32)
        cq.f8_gemm_experts(to_dev(np.stack([wc] * 3)), to_dev(np.stack([ws] * 3)), 2 * n, 512, to_dev(off), xc, xs, act=act, Y=Y)
    else:
        cq.f8_gemm(to_dev(wc), to_dev(ws), 2 * n, 512, xc, xs, act=act, Y=Y)
    got = to_host(Y.float()).astype(np.float64)
    cq.cq_device_error()
    return got


@pytest.mark.parametrize("experts", [False, True])
@pytest.mark.parametrize("n,repeat", [(75, 1), (600, 1), (1300, 12)])
def test_whole_range(n, repeat, experts):
    require_gpu()
    w, x, g, u = _case(n, n)
    plain = _run(w, x, n, repeat, experts, "none", torch.float32)
    g, u = np.tile(g, (repeat, 1)), np.tile(u, (repeat, 1))
    np.testing.assert_array_equal(plain[:, 0::2], g)
    np.testing.assert_array_equal(plain[:, 1::2], u)
    with np.errstate(over="ignore"):
        ref = g / (1 + np.exp(-g)) * u
    top = np.finfo(np.float32).max
    got = _run(w, x, n, repeat, experts, "swiglu", torch.float32)
    big = np.abs(ref) > top * 0.99                         # the largest are infinite in float32
    tol = 17 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -240 * np.abs(u) + 2.0 ** -148
    bad = ~big & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], u[bad][:4], got[bad][:4], ref[bad][:4])
    assert (np.sign(got[big]) == np.sign(ref[big])).all() and (np.abs(got[big]) >= top * 0.98).all()


@pytest.mark.parametrize("seed", [1, 2])
def test_infinite_gates(seed):
    """Gates beyond float32: what the formula gives for the infinities that the plain product shows."""
    require_gpu()
    w, (xc, xs), _, _ = _case(90, seed)
    w[1][:, :3] += 10                                      # gates 2^10 times as large
    plain = _run(w, (xc, xs), 90, 1, False, "none", torch.float32)
    g, u = plain[:, 0::2], plain[:, 1::2]
    assert np.isinf(g).any()
    got = _run(w, (xc, xs), 90, 1, False, "swiglu", torch.float32)
    np.testing.assert_array_equal(np.isnan(got), np.isneginf(g))
    up = np.isposinf(g)
    np.testing.assert_array_equal(got[up], np.sign(u[up]) * np.inf)
