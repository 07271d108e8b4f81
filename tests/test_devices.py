"""(CPU) The F8 and expert-layer calls refuse tensors of different devices, and tensors of a device
that is not the current one: the library launches on the current device, whose kernels would
read memory that is not there."""

import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gemm_cq_gemv_gb300 import _binding

U8, I32, F32, BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


class _OnDevice(torch.Tensor):
    """A host tensor that passes for one of CUDA device `index` (its address is never used)."""
    is_cuda = True
    index = 0

    def get_device(self):
        return self.index


def _fake(index, shape, dtype=F32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)
    t.index = index
    return t


class _Calls:
    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *args: 16
        return lambda *args: self.made.append(name) or 0


# name: call on its tensors, and their shapes and types
CALLS = {
    "f8_quantize": (lambda x, r, c, s, w: cq.f8_quantize(x, rows=r, codes=c, scales=s, workspace=w),
                    [((2, 128), F32), ((3,), I32), ((3, 128), U8), ((3, 4), U8), ((16,), U8)]),
    "f8_quantize_weights": (lambda x, c, s: cq.f8_quantize_weights(x, c, s),
                            [((2, 128), F32), ((2, 128), U8), ((1, 4), U8)]),
    "f8_gemm": (lambda w, ws, x, xs, y: cq.f8_gemm(w, ws, 4, 128, x, xs, Y=y),
                [((4, 128), U8), ((1, 4), U8), ((2, 128), U8), ((2, 4), U8), ((2, 4), F32)]),
    "f8_gemm_experts": (lambda w, ws, o, x, xs, y: cq.f8_gemm_experts(w, ws, 4, 128, o, x, xs, Y=y),
                        [((2, 4, 128), U8), ((2, 1, 4), U8), ((3,), I32), ((2, 128), U8), ((2, 4), U8), ((2, 4), BF16)]),
    "moe_route": (lambda l, w: cq.moe_route(l, 2, workspace=w), [((3, 8), F32), ((16,), U8)]),
    "moe_combine": (lambda y, p, w, o: cq.moe_combine(y, p, w, out=o),
                    [((4, 8), BF16), ((2, 2), I32), ((2, 2), F32), ((2, 8), F32)]),
}


@pytest.fixture
def calls(monkeypatch):
    c, empty = _Calls(), torch.empty
    monkeypatch.setattr(_binding, "_lib", c)
    monkeypatch.setattr(_binding, "_current_device", lambda: 0)
    monkeypatch.setattr(_binding, "_current_stream", lambda device: 0)
    monkeypatch.setattr(_binding, "_raw_stream", _binding._checked_stream)   # as with several devices
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    return c


@pytest.mark.parametrize("name", CALLS)
def test_other_devices_are_refused(name, calls):
    call, specs = CALLS[name]
    call(*(_fake(0, *s) for s in specs))
    assert calls.made == [name]
    for i in range(len(specs)):
        with pytest.raises(ValueError, match="device"):
            call(*(_fake(int(i == j), *s) for j, s in enumerate(specs)))
    with pytest.raises(ValueError, match="not the current one"):
        call(*(_fake(1, *s) for s in specs))
    assert calls.made == [name]
