"""A call on a stream of the caller's: what it allocates is that stream's memory.

Memory of the current stream's pool would be unsafe twice: a block handed out may still be in
use by work queued on the current stream, and a workspace that is dropped when the call
returns may be handed out again there before the kernels have run."""

import contextlib

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gemm_cq_gemv_gb300 import _binding
from gpu_util import require_gpu, to_dev, to_host
from oracle import f8

HANDLE = 0x1230


class _OnDevice(torch.Tensor):
    """A host tensor that passes for a CUDA tensor (its address is never used)."""
    is_cuda = True

    def get_device(self):
        return 0


def _fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


class _Calls:
    """Stands in for the library: every entry point succeeds, every size query asks for 1 KiB."""

    def __getattr__(self, name):
        return lambda *args: 1024 if name.endswith("workspace_bytes") else 0


U8, I8, I16, I32, F32, BF16 = torch.uint8, torch.int8, torch.int16, torch.int32, torch.float32, torch.bfloat16
CALLS = {
    "cq_codebook_fit": (lambda s: cq.cq_codebook_fit(_fake(100, dtype=torch.float64), 4, stream=s), 1),
    "cq_encode": (lambda s: cq.cq_encode(_fake(4, 128), 4, [0.0] * 28, stream=s), 2),
    "a8_quantize": (lambda s: cq.a8_quantize(_fake(2, 128), stream=s), 2),
    "a8_quantize_groups": (lambda s: cq.a8_quantize_groups(_fake(2, 128), 32, stream=s), 2),
    "a8_fake_quant_groups": (lambda s: cq.a8_fake_quant_groups(_fake(2, 128), 32, stream=s), 1),
    "cq_gemv": (lambda s: cq.cq_gemv(_fake(4, 1, 64, dtype=U8), _fake(4, 1, dtype=I16), 4, 128, 4, [0.0] * 28,
                                     _fake(1, 128, dtype=I8), _fake(1), stream=s), 2),
    "cq_gemv_lut": (lambda s: cq.cq_gemv_lut(_fake(4, 1, 32, dtype=U8), _fake(4, 1, dtype=I16), 4, 128, 2, [0.0] * 28,
                                             _fake(1, 128, dtype=I8), _fake(1), stream=s), 1),
    "cq_gemv_noalloc": (lambda s: cq.cq_gemv_noalloc(_fake(4, 1, 64, dtype=U8), _fake(4, 1, dtype=I16), 4, 128, 4,
                                                     [0.0] * 28, _fake(1, 128, dtype=I8), _fake(1), stream=s), 1),
    "cq_gemm": (lambda s: cq.cq_gemm(_fake(4, 1, 64, dtype=U8), _fake(4, 1, dtype=I16), 4, 128, 4, [0.0] * 28,
                                     _fake(9, 128, dtype=I8), _fake(9), stream=s), 2),
    "cq_gemm_grouped": (lambda s: cq.cq_gemm_grouped([], 9, 4, [0.0] * 28, stream=s, device="cpu"), 1),
    "q4_0_quantize": (lambda s: cq.q4_0_quantize(_fake(4, 128), stream=s), 1),
    "q4_0_gemv": (lambda s: cq.q4_0_gemv(_fake(4, 72, dtype=U8), 4, 128, _fake(1, 128), stream=s), 1),
    "q4_0_gemm": (lambda s: cq.q4_0_gemm(_fake(4, 144, dtype=U8), 4, 256, _fake(9, 256), stream=s), 2),
    "f8_quantize": (lambda s: cq.f8_quantize(_fake(1, 128), stream=s), 2),
    "f8_quantize with rows": (lambda s: cq.f8_quantize(_fake(2, 128), rows=_fake(1 << 13, dtype=I32), stream=s), 3),
    "f8_quantize_weights": (lambda s: cq.f8_quantize_weights(_fake(4, 128), stream=s), 2),
    "f8_gemm": (lambda s: cq.f8_gemm(_fake(4, 128, dtype=U8), _fake(1, 4, dtype=U8), 4, 128, _fake(1, 128, dtype=U8),
                                     _fake(1, 4, dtype=U8), stream=s), 1),
    "f8_gemm_experts": (lambda s: cq.f8_gemm_experts(_fake(2, 4, 128, dtype=U8), _fake(2, 1, 4, dtype=U8), 4, 128,
                                                     _fake(3, dtype=I32), _fake(1, 128, dtype=U8),
                                                     _fake(1, 4, dtype=U8), stream=s), 1),
    "moe_route": (lambda s: cq.moe_route(_fake(600, 8), 2, stream=s), 6),
    "moe_combine": (lambda s: cq.moe_combine(_fake(4, 8), _fake(2, 2, dtype=I32), _fake(2, 2), stream=s), 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_stream(name, monkeypatch):
    """(CPU) Every tensor that a call makes is made with the call's stream as the current one, or
    plainly where none is given."""
    current, made, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def record(*args, device=None, **kwargs):
        made.append(current[-1])
        return empty(*args, **kwargs).as_subclass(_OnDevice)

    monkeypatch.setattr(_binding, "_lib", _Calls())
    monkeypatch.setattr(_binding, "_stream", lambda s: s)
    monkeypatch.setattr(_binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    call, tensors = CALLS[name]
    call(HANDLE)
    assert made == [HANDLE] * tensors
    made.clear()
    call(None)
    assert made == [None] * tensors


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_workspaces_on_a_side_stream(handle):
    """The router's and the gather's workspaces while the current stream goes on allocating and
    filling blocks of their sizes, and the side stream is busy before they are used."""
    require_gpu()
    rng = np.random.default_rng(0)
    T, E, k, K = 5000, 64, 4, 1024
    L = to_dev(rng.standard_normal((T, E)).astype(np.float32))
    X = to_dev(rng.standard_normal((T, K)).astype(np.float32))
    want = cq.moe_route(L, k)
    codes, scales = cq.f8_quantize(X, rows=want[3])
    torch.cuda.synchronize()
    sizes = [cq.moe_route_workspace_bytes(T, E), cq.f8_quantize_workspace_bytes(T, K, T * k)]
    assert min(sizes) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    stream = side.cuda_stream if handle else side
    for _ in range(3):
        got = cq.moe_route(L, k, stream=stream)
        c, s = cq.f8_quantize(X, rows=want[3], stream=stream)
        for size in sizes:
            for _ in range(4):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0x3F)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(c, codes) and torch.equal(s, scales)
    rc, rs = f8.f8_quantize(X.cpu().numpy()[:64])
    np.testing.assert_array_equal(to_host(s)[to_host(want[4])[:64, 0]], rs)
    np.testing.assert_array_equal(to_host(c)[to_host(want[4])[:64, 0]], rc)


@pytest.mark.gpu
def test_default_stream_by_handle():
    """Handle 0 is the default stream, not a new one."""
    require_gpu()
    X = torch.randn(40, 300, device="cuda")
    want = cq.f8_quantize(X)
    got = cq.f8_quantize(X, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
