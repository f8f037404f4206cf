"""Quantisation and back on a device that the library is not built for: refused
with GEMM_ERR_ARCH before any launch, as by the other feed-forward operators.
The source is linked against a runtime that reports such a device."""
import ctypes
import os
import subprocess
import sys

import pytest

import shape_adaptive_tile_gb300 as sat

sat_build = sys.modules["shape_adaptive_tile_gb300.build"]

REST = r'''
#include <cuda_runtime.h>
namespace sat {
void set_last_error(const char*) {}
int fail_with(int code, const char*, ...) { return code; }
}  // namespace sat
extern "C" cudaError_t __wrap_cudaGetDevice(int* device) { *device = 0; return cudaSuccess; }
extern "C" cudaError_t __wrap_cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) { *value = 9; return cudaSuccess; }
'''


@pytest.fixture(scope="module")
def elsewhere(tmp_path_factory):
    at = tmp_path_factory.mktemp("elsewhere")
    (at / "rest.cu").write_text(REST)
    subprocess.run([sat_build._nvcc(), *sat_build.FLAGS, "-Xcompiler", "-fno-gnu-unique", "-shared", "-Xlinker", "--wrap=cudaGetDevice",
                    "-Xlinker", "--wrap=cudaDeviceGetAttribute", "-o", str(at / "mxfp4.so"),
                    os.path.join(sat_build.CSRC, "mxfp4.cu"), str(at / "rest.cu")], check=True)
    lib = ctypes.CDLL(str(at / "mxfp4.so"))
    for fn in (lib.mxfp4_quantize, lib.mxfp4_dequantize):
        fn.argtypes = [ctypes.c_void_p] * 2
    return lib


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_is_refused(elsewhere, kind):
    at = 1 << 20
    a = sat.Mxfp4Args(rows=4, width=40, type=kind, values=at, ldv=40, codes=at, ldc=32, scales=at)
    for call in (elsewhere.mxfp4_quantize, elsewhere.mxfp4_dequantize):
        assert call(a.address, None) == -2
    a.rows = 0
    assert elsewhere.mxfp4_quantize(a.address, None) == 0
