"""Build libpagedkv.so in-tree with nvcc for sm_103a (GB300), and _hotcalls.so.

Every translation unit under csrc/ is compiled in parallel, then linked into
one shared library next to this file.  _hotcalls.so (binding/hotcalls.cpp) is the
Python extension that marshals the calls of the shortest kernels; it is compiled
beside the library, against the installed torch, and linked to it.  A user of the C
ABI needs neither torch nor Python's headers: without torch, or with
``python _build.py --library``, the library alone is built.  A stamp of the sources
and flags skips the build when nothing changed.
"""

import hashlib
import importlib.util
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
BINDING_SRC = os.path.join(HERE, "binding", "hotcalls.cpp")
BINDING = os.path.join(HERE, "_hotcalls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", os.path.join(ROOT, "include")]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I",
             os.path.join(ROOT, "include")]


# per-file extra flags (none: the prefill softmax calls the hardware exp2
# through inline PTX, so no unit needs fast-math code generation)
EXTRA_FLAGS = {}


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _sources():
    srcs = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))
    hdrs = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    return srcs, hdrs


def _stamp(srcs, hdrs):
    h = hashlib.sha256()
    for f in srcs + hdrs:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    with open(os.path.join(ROOT, "include", "pagedkv.h"), "rb") as fh:
        h.update(fh.read())
    h.update(" ".join(NVCC_FLAGS + CXX_FLAGS).encode() + repr(sorted(EXTRA_FLAGS.items())).encode())
    return h.hexdigest()


def build_variant(tag, defines, verbose=False):
    """A separate copy of the library compiled with extra -D definitions, for
    tests that need a behaviour the product build must not have (the
    wait-timeout test: a 1 ms wait limit and one decode tile never copied).
    It lands beside the product library as libpagedkv_<tag>.so, from its own
    object directory, and is rebuilt only when sources or definitions change."""
    import fcntl

    lib = os.path.join(HERE, f"libpagedkv_{tag}.so")
    flags = [f"-D{k}={v}" for k, v in sorted(defines.items())]
    with open(lib + ".lock", "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            return _build_locked(False, verbose, lib=lib, build_dir=os.path.join(BUILD, tag),
                                 extra=flags)
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def build(force=False, verbose=False, binding=None):
    """Compile and link the library, and the Python extension unless ``binding`` is
    False (by default it is made where torch is installed, which the Python package
    needs anyway); return the library's path.  Raises on compiler errors.

    Processes that build at the same time (one per rank under torchrun) take
    turns through a lock file next to the library; the later ones find the
    fresh stamp and return at once."""
    import fcntl

    if binding is None:
        binding = importlib.util.find_spec("torch") is not None
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    with open(LIB + ".lock", "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            if not binding:
                return _build_locked(force, verbose)
            with ThreadPoolExecutor(max_workers=1) as ex:
                extension = ex.submit(_compile_binding, force)
                lib = _build_locked(force, verbose)
                _link_binding(*extension.result())
            return lib
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile_binding(force):
    """The binding's object file and the stamp of what it was made from; the object
    is None when the module in place is up to date."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    flags = (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
             + [f"-I{d}" for d in (os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
                                   os.path.join(root, "include"),
                                   os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                   os.path.join(cuda, "include"))])
    h = hashlib.sha256(repr((flags, torch.__version__)).encode())
    for path in (BINDING_SRC, os.path.join(ROOT, "include", "pagedkv.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    stamp = h.hexdigest()
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING + ".stamp"):
        with open(BINDING + ".stamp") as f:
            if f.read().strip() == stamp:
                return None, stamp
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, "hotcalls.cpp.o")
    _run(["g++"] + flags + ["-c", BINDING_SRC, "-o", obj], "compile")
    return obj, stamp


def _link_binding(obj, stamp):
    if obj is None:
        return
    import torch

    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", obj, "-o", tmp,
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda",
          "-ltorch_python", "-L" + HERE, "-lpagedkv", "-Wl,-rpath,$ORIGIN"], "link")
    os.replace(tmp, BINDING)
    with open(BINDING + ".stamp", "w") as f:
        f.write(stamp)


def _build_locked(force, verbose, lib=LIB, build_dir=BUILD, extra=()):
    srcs, hdrs = _sources()
    stamp = _stamp(srcs, hdrs) + ("" if not extra else " " + " ".join(extra))
    stamp_file = lib + ".stamp"
    if not force and os.path.exists(lib) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read().strip() == stamp:
                return lib
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(build_dir, src + ".o")
        path = os.path.join(CSRC, src)
        if src.endswith(".cu"):
            cmd = ([nvcc] + NVCC_FLAGS + EXTRA_FLAGS.get(src, []) + list(extra)
                   + ["-c", path, "-o", obj])
        else:
            cmd = ["g++"] + CXX_FLAGS + list(extra) + ["-c", path, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                binding=False if "--library" in sys.argv else None))
