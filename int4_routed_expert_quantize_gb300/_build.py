"""Build of libcoli_moe.so: nvcc for sm_103a (the host-only tier manager through nvcc's host
compiler), one object per source compiled in parallel."""
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SO = os.path.join(PKG, "libcoli_moe.so")
PY_SO = os.path.join(PKG, "_attn_py.so")  # the attention calls' Python side (csrc/attn_py.cpp), linked to SO
SOURCES = ["pack.cu", "route.cu", "expert_decode.cu", "gateup_w4.cu", "down_w4.cu", "gateup_w8.cu",
           "down_w8.cu", "gateup_w2.cu", "down_w2.cu", "expert_fused.cu", "expert_prefill.cu",
           "runtime.cu", "noalloc.cu", "attn_append.cu", "attn_split.cu", "attn_tile.cu",
           "attn_combine.cu", "attn_runtime.cu", "tier.cpp", "status.cpp"]
HOST_SOURCES = ["tier.cpp", "status.cpp"]  # the parts that need no CUDA


def nvcc_flags(arch="sm_103a"):
    cc = arch.split("_")[1]
    return ["-O3", "-std=c++17", f"-gencode=arch=compute_{cc},code={arch}", "-lineinfo",
            "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def is_stale():
    """True when a library is missing or older than a source or header it is built from"""
    if not os.path.exists(SO) or not os.path.exists(PY_SO):
        return True
    built = min(os.path.getmtime(SO), os.path.getmtime(PY_SO))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + \
        [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > built for p in deps if os.path.isfile(p))


def build(arch="sm_103a", verbose=False, extra=()):
    os.makedirs(BUILD, exist_ok=True)
    flags = nvcc_flags(arch) + list(extra)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = ["nvcc"] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        py = ex.submit(compile_py, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        py_obj = py.result()
    subprocess.check_call(["nvcc", "-shared", "-cudart", "static", "-Xlinker",
                           "--version-script=" + os.path.join(CSRC, "exports.map"), "-o", SO] + objs)
    link_py(py_obj)
    return SO


def compile_py(verbose=False):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "attn_py.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", "/usr/local/cuda/include"]
    cmd += ["-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-c", os.path.join(CSRC, "attn_py.cpp"), "-o", obj]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    return obj


def link_py(obj):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.check_call(["g++", "-shared", "-o", PY_SO, obj, "-L", PKG, "-l:libcoli_moe.so", "-L", lib, "-lc10", "-lc10_cuda",
                           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])


def build_host(out, sanitize=False):
    """Build the host-only parts (tier manager, status strings) with g++ into `out`; with
    `sanitize`, under AddressSanitizer and UndefinedBehaviorSanitizer (for tests)."""
    flags = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC]
    if sanitize:
        flags += ["-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                  "-fno-sanitize-recover=undefined"]
    subprocess.check_call(flags + [os.path.join(CSRC, f) for f in HOST_SOURCES] + ["-o", out])
    return out
