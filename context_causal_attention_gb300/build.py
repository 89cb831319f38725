"""Build libcpattn.so (CUDA, sm_103a) and the Python module of the short calls in-tree under
context_causal_attention_gb300/_build.

Each translation unit is compiled by its own nvcc process in parallel, then
linked into one shared library with the static CUDA runtime.  No cmake.
"""
import concurrent.futures
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libcpattn.so")
BIND = os.path.join(OUT, "_cpbind.so")
TAG = os.path.join(OUT, "_cpbind.tag")
SOURCES = ["attn.cu", "attn_bwd.cu", "attn_tf32.cu", "permute.cu", "merge.cu", "ring.cu", "strategies.cu", "abi.cu",
           "noalloc.cu", "plan.cu", "selftest.cu", "rope.cu", "cache.cu", "prefix.cu", "tree.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _stale(lib, deps):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_tag():
    """What the module is built against: another torch or Python wants another one."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return "torch %s, %s" % (torch, sys.implementation.cache_tag)


def _bind_needs():
    """(root of torch, include paths) for the module, or None and what this machine lacks for it."""
    try:
        import torch
    except ImportError:
        return None, "torch"
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include")]
    for path, header in ((inc[0], "Python.h"), (inc[1], "torch/csrc/autograd/python_variable.h")):
        if not os.path.exists(os.path.join(path, header)):
            return None, header
    if not shutil.which("g++"):
        return None, "g++"
    return root, inc


def _compile_bind(root, inc):
    """bind.cpp against torch's headers, as an object (linked with the library behind it)."""
    import torch

    obj = os.path.join(OUT, "bind.cpp.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
    cmd += ["-isystem" + i for i in inc + [os.path.join(cuda, "include")]]
    cmd += ["-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for bind.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    return [obj, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _link_bind(objects):
    tmp = BIND + ".tmp.%d" % os.getpid()
    link = ["g++", "-shared", "-o", tmp] + objects + ["-L" + OUT, "-lcpattn", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the module failed:\n%s\n%s" % (r.stdout, r.stderr))
    if os.path.exists(TAG):
        os.remove(TAG)  # (never the tag of another module than the one that lies there)
    os.replace(tmp, BIND)
    with open(TAG, "w") as f:
        f.write(_bind_tag())


def _bind_stale(deps):
    if _stale(BIND, deps) or not os.path.exists(TAG):
        return True
    with open(TAG) as f:
        return f.read() != _bind_tag()


def build(force=False, verbose=False):
    """Compile every CUDA source for sm_103a and link libcpattn.so, and the module beside it; returns the library's path.
    The library needs nvcc alone: where torch's headers or Python's are missing, the module is left out (and its
    calls say so), and where the module does not compile, the library stands all the same."""
    os.makedirs(OUT, exist_ok=True)
    header = os.path.join(os.path.dirname(HERE), "include", "cpattn.h")
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(header)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    here = os.path.abspath(__file__)
    lib_stale = force or _stale(LIB, srcs + headers + [here])
    bind_stale = force or _bind_stale([os.path.join(CSRC, "bind.cpp"), header, here])
    if not lib_stale and not bind_stale:
        return LIB
    cc = nvcc() if lib_stale else None
    base = [cc, "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"] + ARCH
    if verbose:
        base += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        cmd = base + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        module = None
        if bind_stale:
            root, needs = _bind_needs()
            if root is None:
                sys.stderr.write("_cpbind.so not built (no %s here): the calls that go through it will raise\n" % needs)
                if os.path.exists(BIND):
                    os.remove(BIND)  # built against something else
            else:
                module = ex.submit(_compile_bind, root, needs)
        results = list(ex.map(compile_one, srcs)) if lib_stale else []
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    if lib_stale:
        tmp = LIB + ".tmp.%d" % os.getpid()
        link = [cc, "-shared"] + ARCH + ["-o", tmp] + [o for o, _ in results] + ["-lpthread"]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    if module is not None:
        _link_bind(module.result())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
