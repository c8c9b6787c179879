"""Build libgbnorm.so in-tree with nvcc for sm_103a (GB300).

Each .cu file is compiled to an object in parallel, then linked into a
shared library next to this file.  No CMake, no torch extension: the library
exports a plain C ABI and is loaded with ctypes, so it does not depend on the
installed PyTorch version.  _block.so next to it is the Python module that
marshals the backbone-block calls (host code compiled against the installed
PyTorch; it calls the same library).

    python -m bwd_bn_pass_gb300.build          # or build_library()
"""

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libgbnorm.so"
MODULE_NAME = "_block.so"
MODULE_SOURCE = "block_py.cpp"

SOURCES = ["abi.cu", "bn_kernels.cu", "rms_kernels.cu", "ln_kernels.cu",
           "row_common.cu", "noalloc.cu", "bn_fused.cu", "bn_small.cu", "fwd_kernels.cu",
           "bn_nhwc.cu", "selftest.cu", "abi_block.cu", "dropout.cu",
           "gn.cu", "rope.cu"]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE,
                "-I", CSRC]


def nvcc_path():
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"),
                 "/usr/local/cuda"):
        if cand:
            p = os.path.join(cand, "bin", "nvcc")
            if os.path.exists(p):
                return p
    p = shutil.which("nvcc")
    if p is None:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return p


def library_path():
    return os.path.join(HERE, LIB_NAME)


def module_path():
    return os.path.join(HERE, MODULE_NAME)


def _module_commands(nvcc):
    """Compile and link commands of the Python module, and its object."""
    import torch
    t = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, os.path.splitext(MODULE_SOURCE)[0] + ".o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    inc = [INCLUDE, os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    compile_ = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                *sum((["-isystem", p] for p in inc), []), "-c",
                os.path.join(CSRC, MODULE_SOURCE), "-o", obj]
    libs = os.path.join(t, "lib")
    link = ["g++", "-shared", "-o", module_path() + ".tmp", obj, "-L", HERE, "-L", libs,
            "-l:" + LIB_NAME, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    return compile_, link


def build_library(verbose=False, extra_flags=()):
    """Compile and link; returns the library path.  Raises on failure."""
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    module_compile, module_link = _module_commands(nvcc)
    procs = [(MODULE_SOURCE, subprocess.Popen(module_compile, stdout=subprocess.PIPE,
                                              stderr=subprocess.STDOUT))]
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH_FLAGS, *COMMON_FLAGS, *extra_flags, "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        msg = "\n".join(f"--- {s} ---\n{t}" for s, t in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    tmp = library_path() + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, library_path())
    r = subprocess.run(module_link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(module_path() + ".tmp", module_path())
    return library_path()


if __name__ == "__main__":
    build_library(verbose="-v" in sys.argv)
    print(library_path())
