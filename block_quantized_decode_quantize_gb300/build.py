"""Build libmemra.so, the sm_103a C-ABI library, in-tree.

Each .cu file under csrc/ is compiled by nvcc in parallel and linked into one shared
library next to this file.  No fast-math: the quantisers rely on IEEE division and
rounding.  csrc/binding.cpp, the Python extension with the quick paths of the small
calls, is compiled against torch's headers at the same time and linked to that library;
where it cannot be built, a warning says why, and the library, which needs no torch, is
there all the same (the Python functions then take their long way to it).
Rebuilds only what has a source or the public header newer than itself.
"""
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings

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


def _newer_than(path, inputs):
    """Whether `path` is there and no input is newer."""
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path)
                                        for f in inputs + [os.path.abspath(__file__)])


def library_up_to_date():
    return _newer_than(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                       glob.glob(os.path.join(INCLUDE, "*.h")))


def binding_up_to_date():
    return _newer_than(BINDING, [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date():
    return library_up_to_date() and binding_up_to_date()


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


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(p, verbose):
    """What a failed command printed, None if it succeeded."""
    out = p.communicate()[0].decode(errors="replace")
    if p.returncode != 0:
        return out or "status %d" % p.returncode
    if verbose and out:
        sys.stderr.write(out)
    return None


def _start_binding(verbose):
    """(started compiler or None, link command, what kept it from starting)."""
    try:
        compile_, link = _binding_cmds()
        return _start(compile_, verbose), link, None
    except Exception as e:  # no torch, no compiler
        return None, None, "%s: %s" % (type(e).__name__, e)


def _finish_binding(p, link, why, verbose):
    if p is not None:
        why = _finish(p, verbose) or _finish(_start(link, verbose), verbose)
    if why is None:
        os.replace(link[link.index("-o") + 1], BINDING)
        return
    if os.path.exists(BINDING):
        os.remove(BINDING)  # of other sources
    warnings.warn("%s is not built; the calls of the cache, attention and routing take their long "
                  "way (14 to 40 us on the host).  The C++ compiler (%s) said:\n%s"
                  % (os.path.basename(BINDING), os.environ.get("CXX", "g++"), why), RuntimeWarning, stacklevel=3)


def build(force=False, verbose=False, extra_flags=()):
    """Compile and link libmemra.so and the Python extension if needed; return the library's path."""
    library = force or not library_up_to_date()
    binding = force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    extension = _start_binding(verbose) if binding else None
    if library:
        procs, objs = [], []
        for src in sources():
            obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
            procs.append((src, _start([nvcc()] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj], verbose)))
            objs.append(obj)
        failed = [(src, why) for src, why in [(src, _finish(p, verbose)) for src, p in procs] if why is not None]
        if failed:
            if extension and extension[0] is not None:
                extension[0].communicate()
            raise RuntimeError("nvcc failed:\n" + "\n".join("%s:\n%s" % f for f in failed))
        tmp = LIB + ".tmp.%d" % os.getpid()
        why = _finish(_start([nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=libmemra.so", "-o", tmp] + objs, verbose),
                      verbose)
        if why is not None:
            raise RuntimeError("linking %s failed:\n%s" % (LIB, why))
        os.replace(tmp, LIB)
    if binding:
        _finish_binding(*extension, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
