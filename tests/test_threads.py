"""Host threads that share a stream and a workspace (CPU): the launches of a
gradient hand each other partial results through the workspace, so no other
call's launch may come between them.

A stand-in for the HIP runtime's entry points, preloaded into a child process,
notes which thread makes each launch, and rests after it so that another thread
would get its turn."""
import os
import shutil
import subprocess
import sys

import pytest

from precision_linear_amd import binding

RUNTIME = r"""
#include <hip/hip_runtime.h>
#include <atomic>
#include <cstring>
#include <unistd.h>
static std::atomic<int> g_count{0};
static int g_caller[1 << 16];
static thread_local int t_caller = -1;
extern "C" {
void note_caller(int id) { t_caller = id; }
int launches(int* out, int n) {
    const int have = g_count.exchange(0);
    for (int i = 0; i < have && i < n; ++i) out[i] = g_caller[i];
    return have;
}
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_t* p, int) {
    memset(p, 0, sizeof(*p));
    strcpy(p->gcnArchName, "gfx950");
    p->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = *block = dim3(1);
    *lds = 0;
    *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t) {
    g_caller[g_count.fetch_add(1) & 0xffff] = t_caller;
    usleep(1000);
    return hipSuccess;
}
}
"""

CHILD = r"""
import ctypes, sys, threading
runtime, path = ctypes.CDLL(sys.argv[1]), sys.argv[2]
L = ctypes.CDLL(path)
P, i64, f32 = ctypes.c_void_p(0x10000), ctypes.c_int64, ctypes.c_float

def linear(ws, M, N, K):
    return L.fp8_linear_backward(P, P, P, 0, P, P, 2, P, P, P, i64(M), i64(N), i64(K), None, ws, i64(1 << 40))

def norm(ws, rows, cols):
    return L.fp8_layer_norm_backward(P, P, 0, P, P, P, 1, None, P, P, P, i64(rows), i64(cols), ws, i64(1 << 40), None)

def taken():
    log = (ctypes.c_int * 65536)()
    return list(log[:runtime.launches(log, 65536)])

# Per-call launches that depend on each other: statistics, quantisation and one or two products; and with
# more column blocks the scales; partial sums and their join, of held and of long rows.
SHAPES = ([(linear, s) for s in ((500, 2048, 2048), (4096, 28672, 8192), (130, 8336, 32))] +
          [(norm, s) for s in ((8191, 1000), (40, 20000))])
same = ctypes.c_void_p(0x700000000000)
alone = {}
for fn, shape in SHAPES:
    runtime.note_caller(0)
    assert fn(same, *shape) == 0
    alone[fn, shape] = len(taken())
    assert alone[fn, shape] >= 2, (fn.__name__, shape, alone[fn, shape])

started = threading.Barrier(len(SHAPES))

def run(number, fn, shape):
    runtime.note_caller(number)
    started.wait()
    for _ in range(5):
        assert fn(same, *shape) == 0

threads = [threading.Thread(target=run, args=(i, *c)) for i, c in enumerate(SHAPES)]
for t in threads: t.start()
for t in threads: t.join()
log = taken()
at = 0
while at < len(log):
    n = alone[SHAPES[log[at]]]
    assert log[at:at + n] == [log[at]] * n, f"launch {at}: calls are mixed: {log[max(0, at - 4):at + 8]}"
    at += n
print("calls kept whole:", at, "launches")
"""


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    rocm = os.path.dirname(os.path.dirname(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")))
    if shutil.which("g++") is None or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("no g++ or HIP headers")
    if not os.path.exists(binding.library_path):
        from precision_linear_amd import build
        build.build()
    d = tmp_path_factory.mktemp("runtime")
    src, lib = str(d / "runtime.cpp"), str(d / "runtime.so")
    with open(src, "w") as f:
        f.write(RUNTIME)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                    src, "-o", lib], check=True)
    return lib


def test_launches_of_one_call_stay_together(runtime):
    r = subprocess.run([sys.executable, "-c", CHILD, runtime, binding.library_path], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=runtime), timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "calls kept whole" in r.stdout
