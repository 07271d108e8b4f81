"""F8 products right behind a long kernel that releases its dependents at its start.

The product's CTAs are then resident while that kernel still runs, for longer than the 2 s after
which the product's own waits give up; its activations are there only at that kernel's end."""

import ctypes
import subprocess

import numpy as np
import pytest
import torch

import gemm_cq_gemv_gb300 as cq
from gemm_cq_gemv_gb300 import build as build_mod
from gpu_util import require_gpu, to_dev, to_host
from oracle import f8

pytestmark = pytest.mark.gpu

SOURCE = r"""
// Releases its dependents, passes `ns` nanoseconds (at most `polls` looks at the clock), copies n bytes.
__global__ void late_copy_kernel(const unsigned char* from, unsigned char* to, long n, unsigned long long ns, long polls) {
    asm volatile("griddepcontrol.launch_dependents;");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (long i = 0; i < polls; ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 >= ns) break;
        __nanosleep(1000);
    }
    __syncthreads();
    for (long i = threadIdx.x; i < n; i += blockDim.x) to[i] = from[i];
}
extern "C" int late_copy(const void* from, void* to, long n, unsigned long long ns, void* stream) {
    late_copy_kernel<<<1, 64, 0, (cudaStream_t)stream>>>((const unsigned char*)from, (unsigned char*)to, n, ns, 1L << 24);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    d = tmp_path_factory.mktemp("late_copy")
    src, so = d / "late_copy.cu", d / "late_copy.so"
    src.write_text(SOURCE)
    subprocess.run([build_mod._nvcc(), *build_mod.ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", str(so), str(src)], check=True)
    fn = ctypes.CDLL(str(so)).late_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_long, ctypes.c_ulonglong, ctypes.c_void_p]

    def call(from_, to, ms):
        assert fn(from_.data_ptr(), to.data_ptr(), to.numel(), int(ms * 1e6), torch.cuda.current_stream().cuda_stream) == 0

    return call


# one tile a CTA, K over a cluster, pairs of CTAs, experts
@pytest.mark.parametrize("M,N,K,E", [(1, 4000, 300, 0), (33, 256, 4096, 0), (400, 2600, 1100, 0), (60, 300, 640, 3)])
@pytest.mark.parametrize("ms", [1, 2500])
def test_product_behind_a_long_kernel(late_copy, M, N, K, E, ms):
    """Exact sums of small integers: one scale, so every product is an integer below 2^24."""
    require_gpu()
    rng = np.random.default_rng(M)
    W = rng.integers(-3, 4, (max(E, 1), N, K)).astype(np.float32)
    X = rng.integers(-3, 4, (M, K)).astype(np.float32)
    wc, ws = cq.f8_quantize_weights(to_dev(W if E else W[0]))
    xc, xs = map(to_dev, f8.f8_quantize(X))
    late = torch.zeros_like(xc)
    Y = torch.full((M, N), float("nan"), device="cuda")
    off = np.linspace(0, M, E + 1).astype(np.int32) if E else None
    off_dev = to_dev(off) if E else None
    torch.cuda.synchronize()
    late_copy(xc, late, ms)
    if E:
        cq.f8_gemm_experts(wc, ws, N, K, off_dev, late, xs, Y=Y)
        want = np.concatenate([X[off[e]:off[e + 1]].astype(np.float64) @ W[e].T.astype(np.float64) for e in range(E)])
    else:
        cq.f8_gemm(wc, ws, N, K, late, xs, Y=Y)
        want = X.astype(np.float64) @ W[0].T.astype(np.float64)
    got = to_host(Y)
    cq.cq_device_error()
    np.testing.assert_array_equal(got, want)
