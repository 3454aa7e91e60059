"""Host side of gq_kv_plan with a CUDA runtime that is none (no GPU needed): a few functions that count their calls.

How many CTAs fit an SM is asked of a cache that all kernels of the library share and that holds a limited number of
(kernel, shared memory) pairs; the lists must not fill it as the number of requests varies."""

import ctypes
import os
import shutil
import subprocess

import pytest

import block_quantized_matvec_gq_gb300 as gq
from block_quantized_matvec_gq_gb300 import build as gqbuild

RUNTIME = r"""
#include <cuda_runtime.h>
static int asked = 0, launched = 0;
static size_t asked_smem = 0, launched_smem = 0;
extern "C" {
int count_asked() { return asked; }
int count_launched() { return launched; }
size_t most_asked() { return asked_smem; }
size_t most_launched() { return launched_smem; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 232448; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *) { *a = cudaFuncAttributes(); return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t smem)
{
    ++asked;
    if (smem > asked_smem) asked_smem = smem;
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **)
{
    ++launched;
    if (c->dynamicSmemBytes > launched_smem) launched_smem = c->dynamicSmemBytes;
    return cudaSuccess;
}
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return 0; }
cudaError_t __cudaGetKernel(void *, const void *) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaSuccess; }
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
}
namespace gq {
int *status_word() { static int word; return &word; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    nvcc = gqbuild.nvcc()
    runtime, obj, so = at / "runtime.cpp", at / "plan.o", at / "plan.so"
    runtime.write_text(RUNTIME)
    subprocess.run([nvcc, *gqbuild.ARCH, *gqbuild.CFLAGS, "-c", os.path.join(gqbuild.CSRC, "gq_plan.cu"), "-o", str(obj)], check=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run([shutil.which("g++"), "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", cuda, str(runtime), str(obj), "-o", str(so)], check=True)
    dll = ctypes.CDLL(str(so))
    dll.most_asked.restype = dll.most_launched.restype = ctypes.c_size_t
    P, I = ctypes.c_void_p, ctypes.c_int
    dll.gq_kv_plan.argtypes = [P] * 11 + [I] * 5 + [P]
    return dll


def test_any_number_of_requests_asks_once(lib):
    A = 1 << 20  # aligned, never dereferenced
    calls = 0
    for n_tokens in (100, 100000):  # in one kernel, and the tokens in a second
        for n_seq in (*range(1, 1500), *range(1500, gq.GQ_MAX_PLAN_SEQ, 97), gq.GQ_MAX_PLAN_SEQ):
            assert lib.gq_kv_plan(*[A] * 11, 4, 4, 16, n_seq, n_tokens, None) == gq.GQ_OK
            calls += 1
    assert lib.count_launched() == calls * 3 // 2
    assert lib.count_asked() == 1
    assert lib.most_asked() >= lib.most_launched() >= 4 * 3 * (gq.GQ_MAX_PLAN_SEQ + 1)
