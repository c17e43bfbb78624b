"""The launchers' once-per-device setting on the host: csrc/q8_launch.h against a fake of the two runtime calls."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q8_quantized_matmul_gb300", "csrc")
FAKE = """
enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidDevice = 101 };
enum cudaFuncAttribute { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
cudaError_t cudaGetDevice(int *d);
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v);
"""
SOURCE = """
#include "q8_launch.h"
static int device, calls, last, result, result_of_get;
cudaError_t cudaGetDevice(int *d) { *d = device; return (cudaError_t)result_of_get; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) { ++calls; last = v; return (cudaError_t)result; }
static q8::SmemAllowed one, two;
extern "C" int allow(int dev, int which, int bytes, int r, int r_get) {
    device = dev; result = r; result_of_get = r_get; calls = 0;
    const cudaError_t e = q8::allow_smem(which ? two : one, &one, bytes);
    return (int)e * 1000 + calls * 100 + (calls ? last : 0);
}
"""


@pytest.fixture(scope="module")
def allow(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    (d / "cuda_runtime.h").write_text(FAKE)
    (d / "launch.cpp").write_text(SOURCE)
    so = str(d / "launch.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", str(d), "-I", CSRC, str(d / "launch.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so).allow


def test_each_device_is_asked_once(allow):
    assert allow(0, 0, 7, 0, 0) == 107 and allow(0, 0, 7, 0, 0) == 0
    assert allow(1, 0, 7, 0, 0) == 107                    # another device of the same process
    assert allow(1, 0, 7, 0, 0) == 0 and allow(0, 0, 7, 0, 0) == 0
    assert allow(1, 1, 9, 0, 0) == 109                    # another kernel
    assert allow(63, 0, 7, 0, 0) == 107 and allow(63, 0, 7, 0, 0) == 0
    assert allow(64, 0, 7, 0, 0) == 107 and allow(64, 0, 7, 0, 0) == 107


def test_errors_are_passed_on_and_asked_again(allow):
    assert allow(5, 0, 7, 1, 0) == 1107 and allow(5, 0, 7, 0, 0) == 107 and allow(5, 0, 7, 0, 0) == 0
    assert allow(6, 0, 7, 0, 101) == 101000


def test_only_the_helper_sets_the_limit():
    """Through allow_smem, or at every call (the routing plan's size differs from call to call)."""
    users = {f for f in os.listdir(CSRC) if "cudaFuncAttributeMaxDynamicSharedMemorySize" in open(os.path.join(CSRC, f)).read()}
    assert users == {"q8_launch.h", "q8_moe.cu"}
