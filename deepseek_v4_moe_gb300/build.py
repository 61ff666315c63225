"""Builds libmoe_ffn.so in the package directory from csrc/*.cu for sm_103a (nvcc, no cmake).

    python -m deepseek_v4_moe_gb300.build [--force]

Each translation unit compiles in parallel into _build/, then one shared library is linked with the
static CUDA runtime (the driver API is reached through cudaGetDriverEntryPointByVersion, so no
libcuda link is needed).  The Python binding of the dense sublayer, _native.so, is compiled beside
them against PyTorch's headers and linked to the library; what it was compiled for is noted beside the
objects, and a binding made for something else is built anew.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_ffn.so")
NATIVE = os.path.join(PKG, "_native.so")
NATIVE_KEY = os.path.join(BUILD, "native.key")
NATIVE_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"]
SOURCES = ["moe_ffn.cu", "prelude.cu", "decode.cu", "decode_tc.cu", "dispatch.cu", "gemm_tc.cu", "splitgemm.cu",
           "noalloc.cu", "dense.cu", "dense_norm.cu", "dense_gemm.cu",
           "dense_fp8.cu", "dense_gemv.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return any(os.path.getmtime(p) > t for p in deps) or not native_fits()


def native_key() -> str:
    """What the binding depends on besides the sources' times: PyTorch (its inline code, types and C++ ABI),
    Python, the compiler's flags, and the interface between the binding and the library."""
    import torch
    digest = hashlib.sha256()
    for path in (os.path.join(INCLUDE, "moe_ffn.h"), os.path.join(CSRC, "binding.cpp")):
        with open(path, "rb") as f:
            digest.update(f.read())
    return "\n".join([f"torch {torch.__version__}", f"cuda {torch.version.cuda}",
                      f"cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"python {sysconfig.get_config_var('SOABI')}",
                      " ".join(NATIVE_FLAGS), digest.hexdigest()])


def native_fits() -> bool:
    """There is a binding, and it was made for this PyTorch, Python and interface."""
    try:
        with open(NATIVE_KEY) as f:
            return os.path.exists(NATIVE) and f.read() == native_key()
    except OSError:
        return False


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_binding(cc: str) -> str:
    import torch
    t = os.path.join(_torch_dir(), "include")
    inc = [INCLUDE, t, os.path.join(t, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(cc)), "include")]
    obj = os.path.join(BUILD, "binding.o")
    cmd = ["g++", *NATIVE_FLAGS,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for p in inc for a in ("-I" if p == INCLUDE else "-isystem", p)],
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    tmp = NATIVE + f".{os.getpid()}.tmp"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libmoe_ffn.so", "-Wl,-rpath,$ORIGIN",
                        "-L", os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
                        "-ltorch_python"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(NATIVE_KEY):  # never the note of one binding beside another
        os.remove(NATIVE_KEY)
    os.replace(tmp, NATIVE)
    tmp = NATIVE_KEY + f".{os.getpid()}.tmp"
    with open(tmp, "w") as f:
        f.write(native_key())
    os.replace(tmp, NATIVE_KEY)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = extra or []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        native = ex.submit(_compile_binding, cc)
        objs = list(ex.map(compile_one, SOURCES))
        binding = native.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
