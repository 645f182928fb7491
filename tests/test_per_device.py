"""Settings that CUDA keeps per device are made on each device, with a stand-in for CUDA (CPU)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "ring_collectives_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include "per_device.h"

static int dev = 0, made[4] = {};
static cudaError_t state = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = dev; return state; }
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main()
{
    rc::OncePerDevice once;
    auto set = [] { ++made[dev]; return cudaSuccess; };
    CHECK(once(set) == cudaSuccess && once(set) == cudaSuccess && made[0] == 1);
    dev = 3;                                        // another device gets its own
    CHECK(once(set) == cudaSuccess && once(set) == cudaSuccess && made[3] == 1 && made[0] == 1);
    dev = 1;                                        // a failure is told and tried again
    CHECK(once([] { return cudaErrorInvalidValue; }) == cudaErrorInvalidValue && once(set) == cudaSuccess && made[1] == 1);
    dev = 0;
    CHECK(once(set) == cudaSuccess && made[0] == 1);
    state = cudaErrorNoDevice;
    CHECK(once(set) == cudaErrorNoDevice);
    printf("ok\n");
    return 0;
}
"""


def test_made_once_on_every_device(tmp_path):
    gxx = shutil.which("g++")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are not available")
    src = tmp_path / "once.cc"
    src.write_text(MAIN)
    exe = str(tmp_path / "once")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", cuda, "-I", CSRC, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def test_no_kernel_attribute_is_set_once_a_process():
    """cudaFuncSetAttribute speaks of the current device: never under a flag of the whole process."""
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path, encoding="utf-8").read()
        assert not re.search(r"static const cudaError_t \w+ = cudaFuncSetAttribute", text), path
        for m in re.finditer(r"call_once\(", text):
            body = text[m.start():text.index("});", m.start())]
            assert "cudaFuncSetAttribute" not in body, path
