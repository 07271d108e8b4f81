"""Gathers of f8_quantize whose indexes repeat: any distribution of them, any time it is called.

The codes and scales are bit-exact (the quantizer has one rounding)."""

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gpu_util import require_gpu, to_dev, to_host
from oracle import f8

pytestmark = pytest.mark.gpu


def _rows(kind, rng, M, R):
    if kind == "even":                                   # every source as often as every other
        return rng.permutation(np.arange(R) % M).astype(np.int32)
    if kind == "one":                                    # all of one source
        return np.full(R, M // 3, np.int32)
    if kind == "none":                                   # every index outside X
        return rng.choice([-1, M, -2 ** 31, 2 ** 31 - 1], R).astype(np.int32)
    if kind == "half":                                   # half of one source, the others at random
        rows = rng.integers(0, M, R)
        return np.where(rng.random(R) < 0.5, M - 1, rows).astype(np.int32)
    return (rng.random(R) ** 6 * (M + 1)).astype(np.int32)   # "steep": few often, some never, some outside


def _check(X, rows, c, s):
    rc, rs = f8.f8_quantize(X)
    M, g = X.shape[0], -(-X.shape[1] // 128)
    inside = (rows >= 0) & (rows < M)
    c, s = to_host(c), to_host(s)
    np.testing.assert_array_equal(s[inside], rs[rows[inside]])
    np.testing.assert_array_equal(c[inside], rc[rows[inside]])
    assert not c[~inside].any() and (s[~inside][:, :g] == 255).all() and (s[~inside][:, g:] == 127).all()


@pytest.mark.parametrize("kind", ["even", "one", "none", "half", "steep"])
@pytest.mark.parametrize("M,K,R,bf16", [(1, 700, 24001, False), (3, 520, 33000, True), (300, 1500, 11190, True),
                                        (5000, 640, 40000, False), (9001, 300, 60000, True)])
def test_any_distribution(kind, M, K, R, bf16):
    require_gpu()
    assert cq.f8_quantize_workspace_bytes(M, K, R) > 0
    rng = np.random.default_rng(M + R)
    X = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32))
    X = X.to(torch.bfloat16) if bf16 else X
    rows = _rows(kind, rng, M, R)
    c, s = cq.f8_quantize(X.cuda(), rows=to_dev(rows))
    _check(X.float().numpy(), rows, c, s)


def test_workspace_is_not_written_past_its_end():
    require_gpu()
    rng = np.random.default_rng(1)
    for M, K, R in ((1, 700, 24001), (300, 1500, 11190), (9001, 300, 60000)):
        X = rng.standard_normal((M, K)).astype(np.float32)
        need = cq.f8_quantize_workspace_bytes(M, K, R)
        for kind in ("even", "one", "none"):
            rows = _rows(kind, rng, M, R)
            space = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
            c, s = cq.f8_quantize(to_dev(X), rows=to_dev(rows), workspace=space[:need])
            _check(X, rows, c, s)
            assert (space[need:] == 0xA5).all()


def _ms(call):
    call()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(3):
        begin.record()
        call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, begin.elapsed_time(end))
    return best


@pytest.mark.parametrize("M", [1, 4000])
@pytest.mark.parametrize("kind", ["one", "none"])
def test_time_does_not_depend_on_the_distribution(M, kind):
    """2^18 rows of one source, or of none, within 20 times of as many rows of distinct sources
    (87 us; one source of 4000 takes 0.1 ms, as a list that one warp walks 29 ms)."""
    require_gpu()
    K, R = 128, 1 << 18
    rng = np.random.default_rng(2)
    X = torch.randn(M, K, device="cuda")
    rows = to_dev(_rows(kind, rng, M, R))
    wide, each = torch.randn(R, K, device="cuda"), to_dev(np.arange(R, dtype=np.int32))
    assert cq.f8_quantize_workspace_bytes(M, K, R) > 0
    assert _ms(lambda: cq.f8_quantize(X, rows=rows)) <= 20 * _ms(lambda: cq.f8_quantize(wide, rows=each))


def test_lists_in_a_graph():
    """A captured gather gives the same bits for new values and new indexes."""
    require_gpu()
    rng = np.random.default_rng(3)
    M, K, R = 3000, 1024, 24000
    X, rows = torch.zeros(M, K, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    codes = torch.empty(R, cq.f8_row_bytes(K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(R, cq.f8_scale_bytes(K), dtype=torch.uint8, device="cuda")
    space = torch.empty(cq.f8_quantize_workspace_bytes(M, K, R), dtype=torch.uint8, device="cuda")
    cq.f8_quantize(X, rows=rows, codes=codes, scales=scales, workspace=space)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cq.f8_quantize(X, rows=rows, codes=codes, scales=scales, workspace=space)
    for kind in ("even", "steep", "half"):
        x, r = rng.standard_normal((M, K)).astype(np.float32), _rows(kind, rng, M, R)
        X.copy_(to_dev(x))
        rows.copy_(to_dev(r))
        graph.replay()
        _check(x, r, codes, scales)
