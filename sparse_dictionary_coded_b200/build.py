"""Build libsdk.so (nvcc for sm_100a) and the Python binding of the calls where
the host's time counts (_binding.so, g++ over torch's headers) in place; no GPU
needed to compile.

    python -m sparse_dictionary_coded_b200.build        # -f: all of it again
    python sparse_dictionary_coded_b200/build.py -c     # the C ABI alone: no torch
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsdk.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_OF = os.path.join(BUILD, "binding.of")   # the Python and torch it was built for

SOURCES = ["api.cu", "chunk_atoms.cu", "chunk_attn.cu", "chunk_direct.cu", "decode.cu", "decode_static.cu", "encode_simt.cu", "encode_small.cu",
           "encode_tc.cu", "out_tc.cu", "paged.cu", "qd_tc.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(obj, src):
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                    if f.endswith(".cuh")] + [os.path.join(ROOT, "include",
                                                           "sdk.h")]
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose=False, force=False, binding=True):
    """Compile every source to an object under _build/ and link libsdk.so;
    with `binding` build _binding.so as well."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    jobs = []
    objs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, src):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj])
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        for cmd, res in zip(jobs, ex.map(
                lambda c: subprocess.run(c, capture_output=True, text=True),
                jobs)):
            if verbose or res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
            if res.returncode != 0:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or jobs or not os.path.exists(LIB):
        # by its name alone, so that _binding.so finds the one beside it wherever they are
        cmd = [nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libsdk.so", "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("link failed")
    if binding:
        build_binding(force)
    return LIB


def binding_stale(src, built_for):
    """Whether _binding.so is missing, older than its source or built for
    another Python or torch, whose headers it was compiled with."""
    if _stale(BINDING, src) or not os.path.exists(BINDING_OF):
        return True
    with open(BINDING_OF) as f:
        return f.read() != built_for


def build_binding(force=False):
    """Compile and link _binding.so against torch and libsdk.so."""
    import sysconfig
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    built_for = "python %s, torch %s at %s\n" % (sys.version, torch.__version__,
                                                os.path.dirname(torch.__file__))
    if not (force or binding_stale(src, built_for)):
        return
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", cuda,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(home, "include"),
           "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           src, "-o", BINDING, "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-L", PKG, "-lsdk", "-L", os.path.join(os.path.dirname(cuda), "lib64"),
           "-lcudart", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed: " + " ".join(cmd))
    with open(BINDING_OF, "w") as f:
        f.write(built_for)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, binding="-c" not in sys.argv))
