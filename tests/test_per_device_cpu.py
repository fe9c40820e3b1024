"""csrc/per_device.h over a runtime that is played: two devices, which refuse and answer differently."""
import os
import shutil
import subprocess

import pytest

import rotated_codebook_quantized_gb300 as tq

CSRC = os.path.join(os.path.dirname(tq.__file__), "csrc")

PLAY = r"""
#include "per_device.h"

#include <cstdio>
#include <cstdlib>

static int device = 0, asked = 0, set_smem = 0, set_wide = 0, occupancy = 0, cleared = 0;
static bool lost = false;

extern "C" {
cudaError_t cudaGetDevice(int* d) {
    *d = device;
    return lost ? cudaErrorNoDevice : cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) {
    ++asked;
    if (d == 7) return cudaErrorInvalidDevice;
    *v = d == 0 ? 152 : 148;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute a, int v) {
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
        ++set_smem;
        return v > 232448 ? cudaErrorInvalidValue : cudaSuccess;
    }
    ++set_wide;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
    ++occupancy;
    if (c->gridDim.x != 16 || c->numAttrs != 1 || c->attrs[0].val.clusterDim.x != 16) std::abort();
    if (device == 2) return cudaErrorInvalidClusterSize;
    *n = device == 0 && c->dynamicSmemBytes <= 200000 ? 4 : 0;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) {
    ++cleared;
    return cudaSuccess;
}
}

#define WANT(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
    int k1 = 0, k2 = 0;
    // multiprocessors: each device's own, asked once; without a device, or an answer, the GB300's
    WANT(tq::device_sms() == 152 && tq::device_sms() == 152 && asked == 1);
    device = 1;
    WANT(tq::device_sms() == 148 && tq::device_sms() == 148 && asked == 2);
    device = 7;
    WANT(tq::device_sms() == 152);
    device = 1, lost = true;
    WANT(tq::device_sms() == 152);
    lost = false, device = 0;
    WANT(tq::device_sms() == 152);
    // shared memory: raised once a device and kernel, and again for more
    WANT(tq::ensure_smem(&k1, 40000) == cudaSuccess && set_smem == 0);
    WANT(tq::ensure_smem(&k1, 100000) == cudaSuccess && tq::ensure_smem(&k1, 90000) == cudaSuccess && set_smem == 1);
    WANT(tq::ensure_smem(&k1, 110000) == cudaSuccess && set_smem == 2);
    WANT(tq::ensure_smem(&k2, 100000) == cudaSuccess && set_smem == 3);
    device = 1;
    WANT(tq::ensure_smem(&k1, 100000) == cudaSuccess && set_smem == 4);
    WANT(tq::ensure_smem(&k1, 300000) != cudaSuccess && tq::ensure_smem(&k1, 300000) != cudaSuccess && set_smem == 6);
    lost = true;
    WANT(tq::ensure_smem(&k1, 100000) != cudaSuccess);
    lost = false, device = 0;
    // clusters: up to 8 without a question; 16 as each device, kernel and size answers
    WANT(tq::clusters_fit(&k1, 8, 512, 100000) && set_wide == 0 && occupancy == 0);
    WANT(tq::clusters_fit(&k1, 16, 512, 100000) && tq::clusters_fit(&k1, 16, 512, 100000) && set_wide == 1 && occupancy == 1);
    WANT(tq::clusters_fit(&k2, 16, 512, 100000) && set_wide == 2);
    WANT(cleared == 0 && !tq::clusters_fit(&k1, 16, 512, 201000) && cleared == 1);
    device = 1;
    WANT(!tq::clusters_fit(&k1, 16, 512, 100000) && !tq::clusters_fit(&k1, 16, 512, 100000) && occupancy == 4);
    device = 2;
    WANT(!tq::clusters_fit(&k1, 16, 512, 100000) && cleared == 3);
    device = 0;
    WANT(tq::clusters_fit(&k1, 16, 512, 100000) && occupancy == 5);
    std::puts("played");
    return 0;
}
"""


def test_what_is_kept_is_kept_by_device(tmp_path):
    include = [d for d in (os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),) if os.path.isdir(d)]
    if not include or not shutil.which("g++"):
        pytest.skip("no compiler, or no CUDA headers")
    src, exe = tmp_path / "play.cpp", tmp_path / "play"
    src.write_text(PLAY)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", CSRC, "-I", include[0], str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "played\n", r.stdout
