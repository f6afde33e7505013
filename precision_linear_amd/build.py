"""Builds libfp8_scaled_mm.so (the HIP kernels -- scaled multiply,
quantiser, layer norm and linear layer -- and their C ABI) for gfx950, and,
where it compiles, _calls.so (the binding's short calls into it, host code).

hipcc cross-compiles without a GPU.  The library is written next to this
file so that it travels with the source tree.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
# The host logic and C ABI, one translation unit per operand-format pair of
# the multiply's kernels (and of those with the linear layer's epilogue), the quantiser, the layer norm
# and the linear layer's gradient.  They compile in parallel.
SRCS = [os.path.join(HERE, "csrc", f) for f in
        ["fp8_scaled_mm.hip"] + [f"fp8_{n}_f{k}.hip" for n in ("gemm", "linear") for k in range(4)] +
        ["fp8_linear_pair.hip", "fp8_quantize.hip", "fp8_layer_norm.hip", "fp8_linear_grad.hip"]]
HEADERS = [os.path.join(HERE, "csrc", f) for f in
           ("fp8_gemm_kernels.h", "fp8_convert.h", "lane_ops.h", "activation.h", "fp8_pair.h",
            "enqueue_lock.h", "plan_cost_table.h")]
LIB = os.path.join(HERE, "libfp8_scaled_mm.so")
# The binding's short calls from torch tensors to the C ABI (host code only).
CALLS_SRC = os.path.join(HERE, "csrc", "torch_calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 VALU forms are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed ({res.returncode}): {' '.join(cmd)}")
    if verbose:
        sys.stderr.write(res.stderr)


# Host-only sanitizer instrumentation (AddressSanitizer + UndefinedBehavior-
# Sanitizer) for the translation units whose host code is the C ABI's logic
# (argument validation, plan and workspace arithmetic); device code is built
# as usual.  Every -fsanitize flag is scoped to the host compilation.
SANITIZE_HOST = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                 "-Xarch_host", "-fno-sanitize-recover=undefined",
                 "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-g"]
HOST_LOGIC_SRCS = {"fp8_scaled_mm.hip", "fp8_quantize.hip", "fp8_layer_norm.hip", "fp8_linear_grad.hip"}


def _calls_command(out):
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "include"),
            *(f"-I{p}" for p in include_paths()), f"-I{sysconfig.get_paths()['include']}", CALLS_SRC,
            f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-ltorch_hip",
            "-o", out]


def _build_calls(out: str, verbose: bool) -> None:
    """Compile _calls to `out` and put it in place.  It only saves host time, so
    where it does not compile (no headers of torch or Python, say) the library is
    built without it, and none of an earlier build stays behind."""
    try:
        _run(_calls_command(out), verbose)
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write(f"_calls is not built, short calls take some microseconds more: {e}\n")
        if os.path.exists(CALLS):
            os.remove(CALLS)
        return
    shutil.move(out, CALLS)


def build(verbose: bool = False, sanitize: bool = False, out: str | None = None) -> str:
    """Compile every source to an object (in parallel), then link the
    shared library; always rebuilds.  sanitize=True builds the host logic
    with ASan/UBSan (a test build, loaded with the sanitizer runtime
    preloaded) into `out` instead of the package's library."""
    from concurrent.futures import ThreadPoolExecutor
    target = out or LIB
    objdir = tempfile.mkdtemp(prefix="fp8mm_build_")
    try:
        objs = [os.path.join(objdir, os.path.basename(src) + ".o") for src in SRCS]
        jobs = []
        for src, obj in zip(SRCS, objs):
            extra = SANITIZE_HOST if sanitize and os.path.basename(src) in HOST_LOGIC_SRCS else []
            jobs.append([HIPCC, *FLAGS, *extra, "-c", src, "-o", obj])
        workers = max(1, min(len(jobs), os.cpu_count() or 1))
        with ThreadPoolExecutor(max_workers=workers) as ex:
            calls = ex.submit(_build_calls, os.path.join(objdir, "_calls.so"), verbose) if out is None else None
            list(ex.map(lambda c: _run(c, verbose), jobs))
            if calls is not None:
                calls.result()
        tmp = target + ".tmp"
        _run([HIPCC, "--offload-arch=gfx950", "-shared", *objs, "-o", tmp], verbose)
        shutil.move(tmp, target)
    finally:
        shutil.rmtree(objdir, ignore_errors=True)
    return target


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
