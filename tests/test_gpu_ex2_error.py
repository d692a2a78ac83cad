"""The largest relative error of ex2.approx.ftz, on which the bound of the draw's FP32 sums
rests: measured over every float of [-125, 125] and compared with the constant that the
kernels use."""
import os
import re
import subprocess

import pytest

from cross_entropy_rl_gb300 import build as B

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <cstring>
__global__ void largest(uint32_t first, uint32_t n, unsigned long long* worst) {
    double m = 0;
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
        const float x = __uint_as_float(first + i);
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        m = fmax(m, fabs(y / exp2(static_cast<double>(x)) - 1.0));
    }
    atomicMax(worst, __double_as_longlong(m));  // numbers from 0 up order as their bits do
}
int main() {
    const float end = 125.f;
    uint32_t last;
    memcpy(&last, &end, 4);
    unsigned long long* worst;
    if (cudaMalloc(&worst, 8) != cudaSuccess || cudaMemset(worst, 0, 8) != cudaSuccess) return 1;
    largest<<<1216, 256>>>(0u, last + 1, worst);
    largest<<<1216, 256>>>(0x80000000u, last + 1, worst);
    double e;
    if (cudaMemcpy(&e, worst, 8, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
    printf("%.6e\n", e);
    return 0;
}
"""


def test_over_all_floats(tmp_path):
    source, program = tmp_path / "ex2.cu", tmp_path / "ex2"
    source.write_text(SOURCE)
    subprocess.run([B.nvcc(), *B.ARCH, "-O3", "-o", str(program), str(source)], check=True)
    worst = float(subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=120).stdout)
    with open(os.path.join(B.ROOT, "cross_entropy_rl_gb300", "csrc", "sample_kernels.cu")) as f:
        used = float(re.search(r"kEx2Error = ([0-9.e-]+);", f.read()).group(1))
    assert 1e-7 < worst <= used
