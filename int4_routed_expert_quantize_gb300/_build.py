"""Build of libcoli_moe.so: nvcc for sm_103a (the host-only tier manager through nvcc's host
compiler), one object per source compiled in parallel."""
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SO = os.path.join(PKG, "libcoli_moe.so")
PY_SO = os.path.join(PKG, "_attn_py.so")  # the attention calls' Python side (csrc/attn_py.cpp), linked to SO
PY_TAG = os.path.join(BUILD, "attn_py.tag")  # what it was built for (torch_tag)
SOURCES = ["pack.cu", "route.cu", "expert_decode.cu", "gateup_w4.cu", "down_w4.cu", "gateup_w8.cu",
           "down_w8.cu", "gateup_w2.cu", "down_w2.cu", "expert_fused.cu", "expert_prefill.cu",
           "runtime.cu", "noalloc.cu", "attn_append.cu", "attn_split.cu", "attn_qsplit.cu", "attn_tile.cu", "attn_qtile.cu",
           "attn_combine.cu", "attn_runtime.cu", "linear.cu", "linear_many.cu", "tier.cpp", "status.cpp"]
HOST_SOURCES = ["tier.cpp", "status.cpp"]  # the parts that need no CUDA


def nvcc_flags(arch="sm_103a"):
    cc = arch.split("_")[1]
    return ["-O3", "-std=c++17", f"-gencode=arch=compute_{cc},code={arch}", "-lineinfo",
            "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def torch_tag():
    """the torch and the Python that _attn_py.so is built for; None where there is no torch (then it is not built)"""
    try:
        import torch
    except ImportError:
        return None
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def is_stale():
    """True when a library is missing, older than a source or header it is built from, or built for another torch"""
    tag, libs = torch_tag(), [SO]
    if tag is not None:
        libs.append(PY_SO)
        if not os.path.exists(PY_TAG) or open(PY_TAG).read() != tag:
            return True
    if not all(os.path.exists(p) for p in libs):
        return True
    built = min(os.path.getmtime(p) for p in libs)
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
        tag = torch_tag()
        py = ex.submit(compile_py, verbose) if tag is not None else None
        objs = list(ex.map(compile_one, SOURCES))
        # the C library first: it needs neither torch nor the Python side
        subprocess.check_call(["nvcc", "-shared", "-cudart", "static", "-Xlinker",
                               "--version-script=" + os.path.join(CSRC, "exports.map"), "-o", SO] + objs)
    if py is not None:
        link_py(py.result())
        with open(PY_TAG, "w") as f:
            f.write(tag)
    return SO


def compile_py(verbose=False):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "attn_py.o")
    # (through nvcc, which knows where the CUDA headers are)
    cmd = ["nvcc", "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-I",
           sysconfig.get_paths()["include"]]
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
