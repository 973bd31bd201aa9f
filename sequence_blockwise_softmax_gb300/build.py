"""Build libra_gb300.so in-tree with nvcc for sm_103a (no torch extension machinery).

Each CUDA translation unit is compiled in parallel, then linked into
``sequence_blockwise_softmax_gb300/_lib/libra_gb300.so`` with the CUDA runtime
linked statically.  Beside it g++ builds ``_lib/ra_torch.<python>-<torch>.so``, the
marshalling of torch tensors for the calls whose host time counts; it holds the
layout of the installed torch's tensors, so its name says which torch that is and
another one builds its own.  Each is rebuilt only when a source or header is
newer.  The library needs nvcc alone: where the binding
cannot be built, the library is there all the same, for callers from C, and then
the failure is raised.
"""
import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libra_gb300.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "ra.h")]


def _newer(path, deps):
    """Whether `path` exists and no dependency is newer."""
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def library_up_to_date():
    return _newer(LIB, _deps())


class BindingError(RuntimeError):
    """The torch binding could not be built; the library was."""


def binding_path():
    """Where the binding for this Python and the installed torch lies."""
    try:
        import torch
    except ImportError as e:
        raise BindingError("the torch binding needs torch: %s" % e)
    tag = "%s-torch%s-%s" % (sys.implementation.cache_tag, torch.__version__, (torch.version.git_version or "")[:12])
    return os.path.join(OUT_DIR, "ra_torch.%s.so" % re.sub(r"[^\w.-]", "_", tag))


def binding_up_to_date():
    try:
        path = binding_path()
    except BindingError:
        return False
    return _newer(path, (BINDING_SOURCE, os.path.join(ROOT, "include", "ra.h")))


def build_binding():
    """Compile the torch binding against the installed torch's headers and libraries."""
    import sysconfig

    path = binding_path()
    import torch
    os.makedirs(OUT_DIR, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + ".%d.tmp" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SOURCE, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise BindingError("g++ did not run for %s: %s" % (BINDING_SOURCE, e))
    if r.returncode != 0:
        raise BindingError("g++ failed for %s:\n%s%s" % (BINDING_SOURCE, r.stdout, r.stderr))
    os.replace(tmp, path)
    return path


def build_library(verbose=False, extra_flags=()):
    os.makedirs(OUT_DIR, exist_ok=True)
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [exe, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"),
               "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(sources()))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [exe, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


def build(force=False, verbose=False, extra_flags=()):
    """The library and the binding side by side; BindingError once the library is there."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = None if not force and binding_up_to_date() else ex.submit(build_binding)
        if force or not library_up_to_date():
            build_library(verbose, extra_flags)
        if binding is not None:
            binding.result()
    return LIB


def main(argv):
    """For callers from C: the library's path; a binding that cannot be built is only reported."""
    v = "-v" in argv
    try:
        build(force=True, verbose=v, extra_flags=["-Xptxas", "-v"] if v else [])
    except BindingError as e:
        print("the library is built, the torch binding is not: %s" % e, file=sys.stderr)
    print(LIB)
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1:]))
