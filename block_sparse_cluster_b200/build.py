"""Build libda.so in-tree with nvcc for sm_100a (one nvcc per source file, in parallel).

    python block_sparse_cluster_b200/build.py [--force]

(Run it by path: importing the package loads libda.so, which this script produces.)
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libda.so")
FAULT_LIB = os.path.join(HERE, "libda_fault.so")
CALL_SRC = os.path.join(CSRC, "layer_call.cpp")
CALL_LIB = os.path.join(HERE, "_layer_call.so")
CALL_STAMP = "layer_call.built_for"   # in BUILD
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-Xptxas", "-warn-spills", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps_mtime():
    files = glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max(os.path.getmtime(f) for f in files)


def _compile(src, extra=()):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r.returncode, r.stdout + r.stderr


def _link(objs, lib):
    r = subprocess.run([NVCC, *ARCH, "-shared", "-o", lib, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc link of {os.path.basename(lib)} failed")


def _cuda_include():
    """CUDA's headers: beside nvcc, which may be a name on PATH or a link, or else those of CUDA_HOME or the usual place."""
    nvcc = shutil.which(NVCC) or NVCC
    homes = [os.path.dirname(os.path.dirname(p)) for p in (os.path.realpath(nvcc), os.path.abspath(nvcc))]
    homes += [os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"]
    dirs = [os.path.join(h, "include") for h in homes if h]
    return next((d for d in dirs if os.path.exists(os.path.join(d, "cuda_runtime.h"))), dirs[0])


def build_call():
    """Compile the layer operators' marshalling module (host code against torch's and Python's headers)."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           *["-I" + d for d in (os.path.join(ROOT, "include"), os.path.join(torch, "include"),
                                os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], _cuda_include())],
           CALL_SRC, "-o", CALL_LIB, "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed: layer_call.cpp")


def _built_for():
    """What the marshalling module is tied to beside its sources: this torch and this Python."""
    version = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py")
    return f"{sysconfig.get_config_var('SOABI')}\n{open(version).read() if os.path.exists(version) else ''}"


def _call_is_current(deps):
    stamp = os.path.join(BUILD, CALL_STAMP)
    return (os.path.exists(CALL_LIB) and os.path.getmtime(CALL_LIB) >= deps and os.path.exists(stamp)
            and open(stamp).read() == _built_for())


def build(verbose=False, force=False, extra=()):
    """Compile every csrc/*.cu for sm_100a and link libda.so, the layer operators' marshalling module
    _layer_call.so, and the test build libda_fault.so (the same sources with DA_FAULT_INJECT defined: one withheld barrier arrival, for the test of
    the bounded device waits); skip what is up to date (the module is not for another torch or Python than it was built for)."""
    os.makedirs(BUILD, exist_ok=True)
    deps = _deps_mtime()
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < deps:
        srcs = sources()
        with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
            results = list(ex.map(lambda s: _compile(s, extra), srcs))
        failed = [r for r in results if r[2] != 0]
        for src, _, rc, log in results:
            if log.strip() and (verbose or rc != 0):
                sys.stderr.write(f"--- {os.path.basename(src)}\n{log}")
        if failed:
            raise RuntimeError("nvcc failed: " + ", ".join(os.path.basename(f[0]) for f in failed))
        _link([r[1] for r in results], LIB)
    if force or not _call_is_current(deps):
        build_call()
        with open(os.path.join(BUILD, CALL_STAMP), "w") as f:
            f.write(_built_for())
    if force or not os.path.exists(FAULT_LIB) or os.path.getmtime(FAULT_LIB) < deps:
        # only the attention kernel differs in the test build
        src = os.path.join(CSRC, "attention_tc.cu")
        obj = os.path.join(BUILD, "attention_tc_fault.o")
        r = subprocess.run([NVCC, *ARCH, *FLAGS, *extra, "-DDA_FAULT_INJECT", "-c", src, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed: attention_tc.cu (fault-injection build)")
        objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in sources()
                if os.path.basename(s) != "attention_tc.cu"]
        _link(objs + [obj], FAULT_LIB)
    return LIB


if __name__ == "__main__":
    t = build(verbose=True, force="--force" in sys.argv)
    print(t)
