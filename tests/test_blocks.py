"""The library's growing device memory, compiled with a stand-in for CUDA's allocator (CPU).

A block that is outgrown is never freed before release: its address may be in a
captured graph or in a launch that another thread is about to make.
"""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include "blocks.h"

static std::set<void *> live;
static size_t room = (size_t)1 << 40, taken = 0;
static int frees = 0;
static bool capturing = false;
static cudaStreamCaptureMode mode_now = cudaStreamCaptureModeGlobal;

extern "C" {
cudaError_t cudaMalloc(void **p, size_t n)
{
    if (capturing && mode_now != cudaStreamCaptureModeRelaxed) return cudaErrorStreamCaptureUnsupported;
    if (taken + n > room) return cudaErrorMemoryAllocation;
    taken += n;
    *p = malloc(16);
    live.insert(*p);
    return cudaSuccess;
}
cudaError_t cudaFree(void *p) { ++frees; live.erase(p); free(p); return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *m)
{
    const cudaStreamCaptureMode x = mode_now;
    mode_now = *m;
    *m = x;
    return cudaSuccess;
}
}

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main()
{
    rc::Block b;
    CHECK(rc::grow(b, 0) == cudaSuccess && !b.ptr);
    CHECK(rc::grow(b, 1) == cudaSuccess && b.bytes == 1 << 20);
    std::set<void *> seen{b.ptr};
    size_t sum = 0;
    for (size_t need = 1; need < ((size_t)1 << 36); need += need / 7 + 1) {
        void *const before = b.ptr;
        const size_t had = b.bytes;
        CHECK(rc::grow(b, need) == cudaSuccess && b.bytes >= need);
        if (b.ptr == before) continue;
        sum += had;
        CHECK(b.old[b.olds - 1] == before && sum <= b.bytes);
        seen.insert(b.ptr);
    }
    CHECK(frees == 0 && live == seen);              // whatever was handed out is still there
    capturing = true;                               // growing inside a capture, and the mode is put back
    void *before = b.ptr;
    CHECK(rc::grow(b, b.bytes + 1) == cudaSuccess && b.ptr != before && mode_now == cudaStreamCaptureModeGlobal);
    capturing = false;
    room = taken + b.bytes + (2 << 20);             // no room for twice the size: the size itself
    before = b.ptr;
    const size_t least = b.bytes + (1 << 20);
    CHECK(rc::grow(b, least) == cudaSuccess && b.bytes == least && b.ptr != before);
    room = taken;                                   // no room at all: nothing changes
    before = b.ptr;
    CHECK(rc::grow(b, least + 1) == cudaErrorMemoryAllocation && b.ptr == before && b.bytes == least);
    CHECK(mode_now == cudaStreamCaptureModeGlobal && live.count(before));
    rc::release(b);
    CHECK(live.empty() && !b.ptr && !b.bytes && !b.olds);
    printf("ok\n");
    return 0;
}
"""


def test_outgrown_memory_stays_until_release(tmp_path):
    gxx = shutil.which("g++")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are not available")
    src = tmp_path / "blocks.cc"
    src.write_text(MAIN)
    exe = str(tmp_path / "blocks")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", cuda, "-I", os.path.join(ROOT, "ring_collectives_gb300", "csrc"), str(src),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
