"""Build libcat.so (the CUDA library behind include/cat.h) in-tree, and the
native marshalling of the Python binding's operator plans beside it.

Each translation unit is compiled by nvcc for sm_103a in parallel, then
linked into ``fft_circulant_attention_gb300/libcat.so``.  The CUDA runtime
is linked statically, so the library depends only on the driver.
``_marshal-<torch version>.so`` is a Python extension without kernels,
compiled against the running torch.
"""
import concurrent.futures as cf
import os
import subprocess
import warnings
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcat.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE,
         "--expt-relaxed-constexpr"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def marshal_path():
    import torch
    return os.path.join(HERE, "_marshal-%s.so" % torch.__version__)


def _build_marshal():
    """Compile the marshalling module.  libcat.so and its other callers do
    without it: where torch, its headers or a C++ compiler are missing, a
    warning says so, and the operator plans of the binding raise when used."""
    try:
        import torch
    except ImportError as e:
        return _no_marshal(e)
    out = marshal_path()
    src = os.path.join(CSRC, "marshal.cpp")
    if os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(src):
        return
    if os.path.exists(out):
        os.remove(out)                       # (never one of an earlier interface)
    import sysconfig
    base = os.path.dirname(torch.__file__)
    tmp = out + ".tmp.%d" % os.getpid()
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I" + sysconfig.get_paths()["include"], *("-isystem" + i for i in inc), src,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return _no_marshal(e)
    if r.returncode != 0:
        return _no_marshal("%s failed for %s:\n%s\n%s" % (cmd[0], src, r.stdout, r.stderr))
    os.replace(tmp, out)


def _no_marshal(why):
    warnings.warn("libcat.so is complete, but AttnPlan, LayerNormPlan and ClipPlan have no "
                  "marshalling module: %s" % why, RuntimeWarning, stacklevel=3)


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files.append(os.path.join(INCLUDE, "cat.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(force=False, verbose=False, extra=()):
    """Compile every .cu under csrc/ and link libcat.so; return its path."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps():
        _build_marshal()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(compile_one, srcs))
        marshal.result()
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
