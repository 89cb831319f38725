"""Build libcpattn.so (CUDA, sm_103a) and the Python module of the short calls in-tree under
context_causal_attention_gb300/_build.

Each translation unit is compiled by its own nvcc process in parallel, then
linked into one shared library with the static CUDA runtime.  No cmake.
"""
import concurrent.futures
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


def _compile_bind():
    """bind.cpp against torch's headers, as an object (linked with the library behind it)."""
    import torch

    root, obj = os.path.dirname(torch.__file__), os.path.join(OUT, "bind.cpp.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
    cmd += ["-isystem" + i for i in inc] + ["-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for bind.cpp:\n%s\n%s" % (r.stdout, r.stderr))
    return [obj, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force=False, verbose=False):
    """Compile every CUDA source for sm_103a and link libcpattn.so, and the module beside it; returns the library's path."""
    os.makedirs(OUT, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "cpattn.h"))
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + headers + [os.path.join(CSRC, "bind.cpp"), os.path.abspath(__file__)]
    if not force and not _stale(LIB, deps) and not _stale(BIND, deps):
        return LIB
    cc = nvcc()
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
        bind = ex.submit(_compile_bind)
        results = list(ex.map(compile_one, srcs))
        bind = bind.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    link = [cc, "-shared"] + ARCH + ["-o", tmp] + [o for o, _ in results] + ["-lpthread"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    tmp = BIND + ".tmp.%d" % os.getpid()
    link = ["g++", "-shared", "-o", tmp] + bind + ["-L" + OUT, "-lcpattn", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the module failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
