"""Products right behind the call that writes their weights, with nothing in between.

The decode products read weights ahead of their wait for the kernel before; the calls that write
weights complete their stores before that.  New weights every time, so that a read of the
previous ones shows."""

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _f8(N, K):
    X = torch.randn(1, K, device="cuda")
    x = cq.f8_quantize(X)
    w = cq.f8_quantize_weights(torch.zeros(N, K, device="cuda"))
    Y = [torch.empty(1, N, device="cuda") for _ in range(2)]

    def write(W):
        cq.f8_quantize_weights(W, *w)

    return write, lambda i: cq.f8_gemm(*w, N, K, *x, Y=Y[i])


def _q4_0(N, K):
    X = torch.randn(1, K, device="cuda")
    blocks = cq.q4_0_quantize(torch.zeros(N, K, device="cuda"))
    Y = [torch.empty(1, N, device="cuda") for _ in range(2)]
    return (lambda W: cq.q4_0_quantize(W, blocks=blocks)), lambda i: cq.q4_0_gemv(blocks, N, K, X, Y=Y[i])


def _cq(product, bits):
    def make(N, K):
        cb = cq.make_codebook(np.linspace(-0.2, 0.2, 28))
        xq, scale = cq.a8_quantize(torch.randn(1, K, device="cuda"))
        packed, norms = cq.cq_encode(torch.zeros(N, K, device="cuda"), bits, cb)
        Y = [torch.empty(1, N, device="cuda") for _ in range(2)]
        return (lambda W: cq.cq_encode(W, bits, cb, packed=packed, norms=norms),
                lambda i: product(packed, norms, N, K, bits, cb, xq, scale, Y=Y[i]))
    return make


CASES = {"f8_gemm": _f8, "q4_0_gemv": _q4_0, "cq_gemv 4": _cq(cq.cq_gemv, 4), "cq_gemv_lut 2": _cq(cq.cq_gemv_lut, 2)}


@pytest.mark.parametrize("N,K", [(512, 512), (4096, 2048)])
@pytest.mark.parametrize("name", CASES)
def test_new_weights_every_time(name, N, K):
    require_gpu()
    write, product = CASES[name](N, K)
    gen = torch.Generator(device="cuda").manual_seed(0)
    W = [torch.randn(N, K, generator=gen, device="cuda") for _ in range(6)]
    for i in range(60):
        write(W[i % 6])
        at_once = product(0)
        torch.cuda.synchronize()
        assert torch.equal(at_once, product(1)), i
    cq.cq_device_error()
