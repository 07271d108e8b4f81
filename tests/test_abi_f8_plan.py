"""f8_gemm_plan refuses what the products refuse, before it looks at the device (CPU)."""

import ctypes

import pytest

import gemm_cq_gemv_gb300 as cq
from gemm_cq_gemv_gb300 import build as build_mod

INV, UNS = 1, 3


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return cq.lib()


def test_plan_validation(lib):
    plan = (ctypes.c_int32 * 3)()

    def f(E, N, K, R, act=0, yt=0, out=plan):
        return lib.f8_gemm_plan(E, N, K, R, act, yt, out)

    assert f(0, 8, 128, 1, out=None) == INV
    for args in ((-1, 8, 128, 1), (0, 0, 128, 1), (0, 8, 0, 1), (0, 8, 128, 0), (0, 8, 128, 1, 2), (0, 8, 128, 1, 0, 2),
                 (0, 9, 128, 1, 1)):
        assert f(*args) == INV, args
    for args in ((1025, 8, 128, 1), (0, (1 << 24) + 1, 128, 1), (0, 8, (1 << 24) + 1, 1), (0, 8, 128, (1 << 30) + 1),
                 (0, 1 << 24, 128, 1 << 30)):
        assert f(*args) == UNS, args


def test_binding_refuses_names():
    with pytest.raises(ValueError):
        cq.f8_gemm_plan(8, 128, 1, act="gelu")
