"""The router in three launches (more than 512 tokens): every size of its chunks, up to several
rounds of the scan over them, against a vectorised float64 form.  Choices and order exact,
weights as in test_parity_moe (2^-18)."""

import numpy as np
import pytest

import gemm_cq_gemv_gb300 as cq
from gpu_util import require_gpu, to_dev, to_host
from oracle import moe

pytestmark = pytest.mark.gpu


def _route(L, k, normalize):
    """oracle.moe.moe_route by sorts."""
    L = np.where(np.isnan(L), -np.inf, L.astype(np.float64))
    T, E = L.shape
    ids = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    best = L.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(L == best, 1.0, np.exp(L - best))
    w = np.take_along_axis(p, ids, axis=1)
    w = w / (w if normalize else p).sum(axis=1, keepdims=True)
    w = np.where(best == -np.inf, 0.0, w)
    order = np.argsort(ids.reshape(-1), kind="stable")
    pos = np.empty(T * k, np.int32)
    pos[order] = np.arange(T * k)
    off = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))]).astype(np.int32)
    return ids, w, off, (order // k).astype(np.int32), pos.reshape(T, k)


def _logits(T, E, k):
    rng = np.random.default_rng(T + E + k)
    L = (2 * rng.standard_normal((T, E)) + rng.standard_normal(E)).astype(np.float32)
    L = np.where(rng.random(L.shape) < 0.05, np.float32(-np.inf), np.round(L * 16) / 16)
    L[T // 3] = -np.inf
    L[T // 2, E // 2] = np.nan
    return L.astype(np.float32)


def test_the_vectorised_form_is_the_oracle():
    for normalize in (False, True):
        L = _logits(60, 9, 3)
        for a, b in zip(_route(L, 3, normalize), moe.moe_route(L, 3, normalize)):
            np.testing.assert_allclose(a, b, rtol=1e-14, atol=0)


# chunks of 16, 17, 33, 54 and 64 tokens; 33 to 1094 chunks, up to 35 of them a scan segment
@pytest.mark.parametrize("T,E,k", [(520, 40, 2), (4097, 64, 8), (4864, 256, 8), (5000, 64, 6), (10000, 31, 4), (16384, 256, 8),
                                   (16383, 600, 2), (19457, 8, 1), (30001, 16, 3), (70000, 10, 2)])
@pytest.mark.parametrize("normalize", [False, True])
def test_many_tokens(T, E, k, normalize):
    require_gpu()
    L = _logits(T, E, k)
    got = [to_host(x) for x in cq.moe_route(to_dev(L), k, normalize=normalize)]
    ref = _route(L, k, normalize)
    for i in (0, 2, 3, 4):
        np.testing.assert_array_equal(got[i], ref[i])
    assert (np.abs(got[1] - ref[1]) <= 2.0 ** -18 * ref[1] + 2.0 ** -126).all()
