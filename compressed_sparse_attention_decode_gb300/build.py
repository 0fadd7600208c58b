"""Build libcsa2.so in-tree: one nvcc process per translation unit, in
parallel, for sm_103a only, then one shared-library link; and next to it
_native.so, the part of the Python binding that is written in C++."""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcsa2.so")
NATIVE = os.path.join(HERE, "_native.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
         "--Werror", "cross-execution-space-call",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", os.path.join(HERE, "..", "include")]


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    deps = [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(HERE, "..", "include", "*.h"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _binding():
    """the C++ part of the binding: host code only, against PyTorch's and Python's own headers"""
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src] + glob.glob(os.path.join(HERE, "..", "include", "*.h"))
    import sysconfig

    import torch
    made_for = "%s %s %s" % (sys.version, torch.__version__, torch.__file__)
    stamp = os.path.join(BUILD, "native_made_for")
    if (os.path.exists(NATIVE) and os.path.getmtime(NATIVE) >= max(os.path.getmtime(d) for d in deps)
            and _read(stamp) == made_for):
        return NATIVE
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"]]
    tmp = NATIVE + ".%d.tmp" % os.getpid()
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
           + ["-I" + i for i in inc] + [src, "-o", tmp, "-L" + os.path.join(root, "lib")]
           + ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    os.replace(tmp, NATIVE)
    with open(stamp, "w") as f:
        f.write(made_for)
    return NATIVE


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".%d.tmp" % os.getpid()
        subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    binding.result()                             # its failure is told after the library is there
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
