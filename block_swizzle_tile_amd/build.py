"""Build the gfx950 HIP library libbst.so in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = ["bst.hip", "inst_f16.hip", "inst_bf16.hip", "inst_i8.hip", "inst_fp8.hip",
           "inst_mxfp8.hip", "inst_slicek.hip", "block.hip", "block_gemm_plain_t.hip",
           "block_gemm_plain_n.hip", "block_gemm_grouped_t.hip", "block_gemm_grouped_n.hip",
           "block_grad.hip"]
HEADERS = ["bst_device.hpp", "bst_kernel_dma.hpp", "bst_instances.hpp", "bst_block.hpp",
           "bst_block_gemm.hpp", "bst_block_grad.hpp", "bst_block_quant.hpp",
           "bst_block_rows.hpp", "bst_block_instances.hpp"]
DEPS = ([os.path.join(CSRC, f) for f in SOURCES + HEADERS] +
        [os.path.join(ROOT, "include", f) for f in ("bst.h", "bst_block.h")])
LIB = os.path.join(PKG, "libbst.so")
# The short way from Python to the block-scaled operators: host code only,
# against torch's and Python's headers, so its file is named after both
# (_lib.fast_path).  libbst.so needs neither.
FAST_SOURCE = os.path.join(CSRC, "block_fast.cpp")
# The same kernels with cycle accounting (-DBST_TRACE): per-wave K-loop and
# task phase cycles of workgroup 0 and a per-workgroup shader-clock record,
# written to a device buffer set with bst_debug_set_trace.  For measurement
# only; bench.py --clock loads it.
TRACE_LIB = os.path.join(PKG, "libbst_trace.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-pass-failed",
]


def build(force: bool = True, verbose: bool = False, trace: bool = False) -> str:
    """Compile libbst.so (always when force, else only when a source is newer), which takes hipcc
    alone, and _block_fast for the torch that is importable, if any: a failure of that is raised
    after libbst.so is in place.  trace=True builds libbst_trace.so instead."""
    lib = TRACE_LIB if trace else LIB
    fast = _start_fast(force) if not trace else None
    if not force and os.path.exists(lib) and all(
            os.path.getmtime(lib) >= os.path.getmtime(d) for d in DEPS):
        _finish_fast(fast)
        return lib
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    objdir = os.path.join(PKG, "_build_trace" if trace else "_build")
    flags = HIPCC_FLAGS + (["-DBST_TRACE"] if trace else [])
    os.makedirs(objdir, exist_ok=True)
    procs = []
    for src in SOURCES:     # one process per translation unit, in parallel
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        cmd = ([hipcc] + flags + ["-I", os.path.join(ROOT, "include"), "-c",
                                  os.path.join(CSRC, src), "-o", obj])
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    objs, failed = [], False
    for obj, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            sys.stderr.write(out)
            failed = True
        objs.append(obj)
    if failed:
        raise RuntimeError("hipcc failed building " + os.path.basename(lib))
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("linking %s failed" % os.path.basename(lib))
    os.replace(tmp, lib)
    _finish_fast(fast)
    return lib


def _start_fast(force):
    """Starts compiling _block_fast: (file, temporary file, process).  None if it is up to date or
    there is no torch to bind; a text if it cannot be started."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        print("torch is not importable (%s): _block_fast is not built" % e, file=sys.stderr)
        return None
    from ._lib import fast_path
    out = fast_path(torch.__version__)
    deps = [FAST_SOURCE] + [os.path.join(ROOT, "include", f) for f in ("bst.h", "bst_block.h")]
    if not force and os.path.exists(out) and all(
            os.path.getmtime(out) >= os.path.getmtime(d) for d in deps):
        return None
    import sysconfig

    tmp = out + ".tmp%d" % os.getpid()
    inc = cpp_extension.include_paths() + ["/opt/rocm/include", sysconfig.get_paths()["include"],
                                           os.path.join(ROOT, "include")]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] +
           [x for i in inc for x in ("-isystem" if "torch" in i else "-I", i)] +
           [FAST_SOURCE, "-o", tmp, "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch_hip", "-lc10_hip", "-lc10"])
    try:
        pr = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        return str(e)
    return out, tmp, pr


def _finish_fast(started):
    if started is None:
        return
    if isinstance(started, str):
        raise RuntimeError("_block_fast was not built: " + started)
    lib, tmp, pr = started
    out, _ = pr.communicate()
    if pr.returncode != 0:
        sys.stderr.write(out)
        raise RuntimeError("g++ failed building " + os.path.basename(lib))
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(verbose=True, trace="--trace" in sys.argv[1:]))
