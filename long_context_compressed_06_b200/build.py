"""Build libcsa.so in-tree (sm_100a) with nvcc.

Each .cu under csrc/ is compiled to an object in _build/ (parallel, skipped
when up to date) and linked into long_context_compressed_06_b200/libcsa.so
against the shared CUDA runtime.  csrc/binding_native.cpp, the C++ side of the
binding, is then compiled with g++ against torch's headers into _native.so beside
it; where that cannot be done the binding does without, and a line says so.
"""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libcsa.so")
NATIVE_SRC, NATIVE = os.path.join(CSRC, "binding_native.cpp"), os.path.join(PKG, "_native.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                 "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _deps_mtime(src: str) -> float:
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in headers])


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= _deps_mtime(src):
        return obj
    cmd = [NVCC] + CFLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def build_native(force: bool = False) -> str:
    import shutil
    import sysconfig

    import torch
    # (built against these headers: another torch or interpreter means another file)
    stamp, now = os.path.join(BUILD, "_native.stamp"), "%s %s" % (torch.__version__, sys.version)
    if (not force and os.path.exists(NATIVE) and os.path.exists(stamp) and open(stamp).read() == now
            and os.path.getmtime(NATIVE) >= _deps_mtime(NATIVE_SRC)):
        return NATIVE
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    nvcc = shutil.which(NVCC) or NVCC  # (a path, or a name to look up)
    cuda = [os.path.dirname(os.path.dirname(p)) for p in (nvcc, os.path.realpath(nvcc))]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(),
           '-DCSA_TORCH_VERSION="%s"' % torch.__version__, "-I", os.path.join(ROOT, "include")]
    for d in [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]] + \
            [os.path.join(c, "include") for c in cuda]:
        cmd += ["-isystem", d]
    cmd += [NATIVE_SRC, "-o", NATIVE + ".tmp", "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (NATIVE_SRC, r.stdout, r.stderr))
    os.replace(NATIVE + ".tmp", NATIVE)
    with open(stamp, "w") as f:
        f.write(now)
    return NATIVE


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    lib = _build_lib(force, verbose)
    try:
        build_native(force)
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write("_native.so is not built, the binding does without it: %s\n" % e)
    return lib


def _build_lib(force: bool, verbose: bool) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs)):
        return LIB
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "shared", "-o", LIB + ".tmp"] + objs + \
        ["-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
