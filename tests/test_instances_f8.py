"""Every instance of the F8 product kernel against the float64 product.

Which instance a call takes is the library's estimate, so the sizes here are checked, all together,
to reach every one of them: 16 to 128 tokens a tile with and without K split over a cluster,
pairs of CTAs with tiles of up to 224 and 256 tokens, for experts too.  Tolerances as in
test_parity_f8; codes are random over all of e4m3, scales over 32 powers of two."""

import functools

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gpu_util import require_gpu, to_dev, to_host
from oracle import f8
from test_parity_f8 import _check

pytestmark = pytest.mark.gpu

KINDS = {"f32": ("none", torch.float32), "bf16": ("none", torch.bfloat16), "f32 gated": ("swiglu", torch.float32),
         "bf16 gated": ("swiglu", torch.bfloat16)}

# M, N, K.  Single CTAs take several tiles each where K is not split, pairs too; those of 256 tokens
# (two accumulators that share columns) with one run of K, with two and with three (float32)
DENSE = [(13, 26001, 515), (30, 26001, 1100), (60, 24001, 700), (128, 20001, 700),
         (97, 520, 1536), (147, 66, 910), (3, 64, 913), (700, 68, 2050), (330, 68, 1400), (160, 74, 2700),
         (1265, 134, 3300), (1310, 70, 3608), (318, 70, 7154), (69, 3280, 5000), (1332, 146, 8199), (66, 1554, 10429),
         (500, 13001, 520), (300, 14001, 2500),
         (711, 12110, 1844), (1000, 9001, 4096), (1846, 4151, 4500), (1000, 12801, 5000)]
# R, E, N, K
EXPERTS = [(40, 3, 20001, 310), (620, 2, 70, 1950), (310, 2, 74, 1400), (8, 2, 66, 930), (2590, 3, 66, 320),
           (2590, 3, 70, 3400), (1310, 2, 72, 3900), (345, 2, 80, 5009), (4040, 5, 270, 320), (3909, 11, 140, 4924),
           (2600, 3, 66, 8258), (3000, 6, 2113, 2500), (9000, 40, 2050, 520)]


def _even(N, act):
    return N + (N & 1 if act == "swiglu" else 0)


def _instance(M, N, K, E, kind):
    """The kernel instance of a call: tokens a tile, pairs, K split."""
    act, dtype = KINDS[kind]
    tokens, ctas, split = cq.f8_gemm_plan(_even(N, act), K, M, experts=E, act=act, dtype=dtype)
    if ctas == 2:
        tokens = 256 if tokens > 224 else 224
    return tokens, ctas == 2, split > 1


def test_sizes_reach_every_instance():
    require_gpu()
    single = {(bt, False, split) for bt in (16, 32, 64, 128) for split in (False, True)}
    dense = {_instance(*s, 0, kind) for s in DENSE for kind in KINDS}
    assert dense == single | {(224, True, False), (256, True, False)}
    experts = {_instance(R, N, K, E, kind) for R, E, N, K in EXPERTS for kind in KINDS}
    assert experts == {i for i in single if i[0] > 16} | {(224, True, False)}
    # the shared accumulator columns: one run of K, an even and an odd number, more tiles than pairs
    runs = {-(-K // 2048) for M, N, K in DENSE if _instance(M, N, K, 0, "f32") == (256, True, False)
            and -(-M // 256) * -(-N // 256) > torch.cuda.get_device_properties(0).multi_processor_count // 2}
    assert runs >= {1, 3} and any(r % 2 == 0 for r in runs)


def _codes(rng, *shape):
    c = rng.integers(0, 254, shape).astype(np.uint8)
    return np.where(c >= 0x7F, c + 1, c).astype(np.uint8)          # all but 0x7F and 0xFF, the NaN


def _rows(rng, lead, rows, scale_rows, K, low):
    g = -(-K // 128)
    codes = _codes(rng, *lead, rows, 128 * g)
    codes[..., K:] = 0
    scales = np.full((*lead, scale_rows, cq.f8_scale_bytes(K)), 127, np.uint8)
    scales[..., :g] = rng.integers(low, low + 6, (*lead, scale_rows, g))
    return codes, scales


def _values(codes, scales):
    """float64 values on the GPU; scales per row of codes."""
    table = torch.from_numpy(f8.e4m3_values()).cuda()
    g = codes.shape[-1] // 128
    v = table[to_dev(codes).long()].view(*codes.shape[:-1], g, 128)
    s = torch.exp2(to_dev(scales[..., :g].astype(np.float64)) - 127)
    return (v * s[..., None]).view(codes.shape)


def _product(wc, ws, xc, xs):
    x, w = _values(xc, xs), _values(wc, ws.repeat(128, axis=0)[: wc.shape[0]])
    return to_host(x @ w.T), to_host(x.abs() @ w.abs().T)


@functools.lru_cache(maxsize=1)   # the kinds of a size follow one another
def _dense(M, N, K):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    w, x = _rows(rng, (), N, -(-N // 128), K, 113), _rows(rng, (), M, M, K, 116)
    return w, x, _product(*w, *x)


@functools.lru_cache(maxsize=1)
def _experts(R, E, N, K):
    rng = np.random.default_rng(R * 31 + N * 7 + K + E)
    off = np.sort(np.concatenate([[0, R], (rng.random(E - 1) ** 2 * R).astype(np.int64)])).astype(np.int32)
    w, x = _rows(rng, (E,), N, -(-N // 128), K, 113), _rows(rng, (), R, R, K, 116)
    parts = [_product(w[0][e], w[1][e], x[0][a:b], x[1][a:b]) for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a]
    return w, x, off, tuple(np.concatenate(p) for p in zip(*parts))


def _compare(Y, ref, K, kind):
    got = to_host(Y.float()).astype(np.float64)
    cq.cq_device_error()
    _check(got, *ref, 128 * -(-K // 128), KINDS[kind][0], KINDS[kind][1] == torch.float32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K, kind):
    require_gpu()
    act, dtype = KINDS[kind]
    w, x, ref = _dense(M, _even(N, "swiglu"), K)
    N = _even(N, act)
    w = (w[0][:N], w[1])
    Y = torch.full((M, N // 2 if act == "swiglu" else N), float("nan"), device="cuda", dtype=dtype)
    cq.f8_gemm(*map(to_dev, w), N, K, *map(to_dev, x), act=act, Y=Y)
    _compare(Y, [r[:, :N] for r in ref], K, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,E,N,K", EXPERTS)
def test_experts(R, E, N, K, kind):
    require_gpu()
    act, dtype = KINDS[kind]
    w, x, off, ref = _experts(R, E, _even(N, "swiglu"), K)
    N = _even(N, act)
    w = (w[0][:, :N], w[1])
    Y = torch.full((R, N // 2 if act == "swiglu" else N), float("nan"), device="cuda", dtype=dtype)
    cq.f8_gemm_experts(*map(to_dev, w), N, K, to_dev(off), *map(to_dev, x), act=act, Y=Y)
    _compare(Y, [r[:, :N] for r in ref], K, kind)
