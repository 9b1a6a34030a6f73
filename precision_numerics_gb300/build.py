"""Build the CUDA library libattn.so in-tree with nvcc (sm_103a only).

Each .cu file under csrc/ is compiled in parallel to an object under
_build/, then linked into precision_numerics_gb300/_lib/libattn.so with the
CUDA runtime linked statically.  build_test_variant() makes the test build
(_lib/libattn_testhooks.so, objects under _build_testhooks/), which only the
test suite loads.  A rebuild happens when any source or
header is newer than the library.

csrc/torch_calls.cpp becomes the Python module _lib/_attn_torch.<torch version>.so
(g++ against the installed PyTorch's headers, linked to libattn.so beside it), the
serving calls' binding.  The library needs neither it nor PyTorch: a module that
cannot be built is reported as a warning, and the serving calls go through ctypes,
as all others do.
"""
from __future__ import annotations

import contextlib
import fcntl
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libattn.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_calls.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


# The test build: the same sources with test-only instrumentation compiled in
# (ATTN_TEST_HOOKS: counters and a stall switch in the forward kernel) and a
# 50 ms limit on every in-kernel wait.  Only the test suite loads it.
TEST_VARIANT = "testhooks"
TEST_FLAGS = ("-DATTN_TEST_HOOKS", "-DATTN_TEST_WAIT_LIMIT_NS=50000000ull")


def lib_path(variant: str = "") -> str:
    return LIB if not variant else os.path.join(LIB_DIR, f"libattn_{variant}.so")


def binding_path() -> str:
    """The tensor binding of the installed PyTorch (another version has another ABI)."""
    import torch
    return os.path.join(LIB_DIR, f"_attn_torch.{torch.__version__}.so")


def _older(lib, inputs) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in inputs)


def _binding_needs_build() -> bool:
    try:
        path = binding_path()
    except ImportError:  # no PyTorch, nothing to bind to
        return False
    return _older(path, [BINDING_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h")), os.path.abspath(__file__)])


def needs_build(variant: str = "") -> bool:
    return _older(lib_path(variant), _inputs()) or (not variant and _binding_needs_build())


@contextlib.contextmanager
def _build_lock():
    """Exclusive lock on _lib/.build.lock: processes that build at the same time
    (one per rank under torchrun, say) take turns, so none links objects that
    another one is still writing."""
    os.makedirs(LIB_DIR, exist_ok=True)
    with open(os.path.join(LIB_DIR, ".build.lock"), "w") as fh:
        fcntl.flock(fh, fcntl.LOCK_EX)
        try:
            yield
        finally:
            fcntl.flock(fh, fcntl.LOCK_UN)


def build(force: bool = False, verbose: bool = False, extra_flags=(), variant: str = "") -> str:
    """Compile and link libattn.so (or libattn_<variant>.so); returns its path."""
    lib = lib_path(variant)
    if not force and not needs_build(variant):
        return lib
    with _build_lock():
        # Another process may have built it while this one waited for the lock.
        if not force and not needs_build(variant):
            return lib
        return _build_locked(lib, verbose, extra_flags, variant, force)


def _build_locked(lib, verbose, extra_flags, variant, force=False) -> str:
    nvcc = _nvcc()
    build_dir = BUILD if not variant else BUILD + "_" + variant
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}\n{r.stdout}")
        if verbose and (r.stderr.strip() or r.stdout.strip()):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = None
        if not variant and (force or _binding_needs_build()):
            binding = ex.submit(_compile_binding, build_dir)
        if force or _older(lib, _inputs()):
            objs = list(ex.map(compile_one, srcs))
            tmp = f"{lib}.tmp{os.getpid()}"
            _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], f"link of {os.path.basename(lib)}")
            os.replace(tmp, lib)
    if binding is not None:
        try:
            _link_binding(binding.result())
        except (OSError, ImportError, RuntimeError) as e:
            warnings.warn(f"the tensor binding was not built, the serving calls go through ctypes: {e}", RuntimeWarning,
                          stacklevel=3)
    return lib


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}\n{r.stdout}")


def _compile_binding(build_dir) -> str:
    obj = os.path.join(build_dir, "torch_calls.cpp.o")
    include = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    _run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
          "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", BINDING_SOURCE, "-o", obj],
         "g++ on torch_calls.cpp")
    return obj


def _link_binding(obj) -> None:
    path = binding_path()
    tmp = f"{path}.tmp{os.getpid()}"
    _run([os.environ.get("CXX") or "g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libattn.so",
          "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-ltorch_cuda", "-lc10", "-lc10_cuda"], "link of the tensor binding")
    os.replace(tmp, path)


def build_test_variant(force: bool = False) -> str:
    """The test build (TEST_FLAGS) as _lib/libattn_testhooks.so; returns its path."""
    return build(force=force, extra_flags=TEST_FLAGS, variant=TEST_VARIANT)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
