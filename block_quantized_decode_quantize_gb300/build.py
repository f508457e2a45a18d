"""Build libmemra.so, the sm_103a C-ABI library, in-tree.

Each .cu file under csrc/ is compiled by nvcc in parallel and linked into one shared
library next to this file.  No fast-math: the quantisers rely on IEEE division and
rounding.  csrc/binding.cpp, the Python extension with the quick paths of the small
calls, is compiled against torch's headers at the same time and linked to that library.
Rebuilds only when a source or the public header is newer than the libraries.
"""
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmemra.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_memra_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
                     "-Wall", "-I" + INCLUDE, "-I" + CSRC]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [BINDING_SRC] +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date():
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _binding_cmds():
    """(compile, link) commands of the Python extension."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    obj = os.path.join(BUILD_DIR, "binding.o")
    inc = os.path.join(torch_dir, "include")
    compile_ = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE,
                "-I" + sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
                os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
                os.path.join(cuda, "include"), "-c", BINDING_SRC, "-o", obj]
    libs = os.path.join(torch_dir, "lib")
    link = [os.environ.get("CXX", "g++"), "-shared", "-o", BINDING + ".tmp.%d" % os.getpid(), obj,
            LIB, "-L" + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    return compile_, link


def build(force=False, verbose=False, extra_flags=()):
    """Compile and link libmemra.so if needed; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc()] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT)))
        objs.append(obj)
    compile_binding, link_binding = _binding_cmds()
    if verbose:
        print(" ".join(compile_binding), file=sys.stderr)
    procs.append((BINDING_SRC, subprocess.Popen(compile_binding, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            sys.stderr.write(out.decode(errors="replace"))
    if failed:
        msg = "\n".join("%s:\n%s" % f for f in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=libmemra.so", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    if verbose:
        print(" ".join(link_binding), file=sys.stderr)
    subprocess.run(link_binding, check=True)
    os.replace(BINDING + ".tmp.%d" % os.getpid(), BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
