"""Build the CUDA library (librar.so) in-tree with nvcc for sm_103a, and the
module that calls its model operators on torch tensors (_torch_ops.so) with g++.

Each translation unit compiles in its own process, in parallel, then one
link step makes the shared library.  IEEE behaviour is kept (no fast-math,
no FMA contraction, no flush-to-zero)."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "librar.so")
TORCH_OPS_PATH = os.path.join(BUILD_DIR, "_torch_ops.so")

SOURCES = ["rar_api.cu", "fused.cu", "fused_stream.cu", "ring.cu", "ll.cu", "tree.cu", "noalloc.cu",
           "rmsnorm.cu", "rmsnorm_grad.cu", "vocab_xent.cu", "vocab_logprobs.cu", "embedding.cu", "grad_norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-ftz=false", "-prec-div=true",
              "-prec-sqrt=true", "-fmad=false", "-Xptxas", "-warn-spills", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "rar.h"))
    return files


def up_to_date() -> bool:
    outputs = [LIB_PATH] + ([] if binding_lacks() else [TORCH_OPS_PATH])
    if not all(os.path.exists(f) for f in outputs):
        return False
    if len(outputs) > 1 and _built_against() != _torch_version():
        return False
    t = min(os.path.getmtime(f) for f in outputs)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _torch_dir() -> str | None:
    """Where torch is installed (it is not imported)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_version() -> str:
    """The torch and Python that the binding's ABI belongs to."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        version = next((line.split("=")[1].strip(" '\"\n") for line in f if line.startswith("__version__")), "")
    return f"{version} in {_torch_dir()}, {sysconfig.get_config_var('EXT_SUFFIX')}"


def _built_against() -> str | None:
    try:
        with open(TORCH_OPS_PATH + ".torch") as f:
            return f.read()
    except FileNotFoundError:
        return None


def _cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(shutil.which(_nvcc()) or _nvcc())), "include")


def binding_lacks() -> str | None:
    """What the module on torch tensors needs, beyond what the library needs,
    and this machine does not have; None where it can be built."""
    torch_dir = _torch_dir()
    if not torch_dir:
        return "torch"
    if not shutil.which("g++"):
        return "g++"
    needs = [os.path.join(sysconfig.get_paths()["include"], "Python.h"),
             os.path.join(torch_dir, "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(torch_dir, "include", "c10", "cuda", "CUDAStream.h"),
             os.path.join(torch_dir, "lib", "libtorch_python.so"),
             os.path.join(torch_dir, "lib", "libc10_cuda.so"),
             os.path.join(_cuda_include(), "cuda_runtime_api.h")]
    return next((f for f in needs if not os.path.exists(f)), None)


def _compile_torch_ops(obj: str) -> None:
    torch_dir = _torch_dir()
    cuda = _cuda_include()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(torch_dir, "include"), "-isystem",
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-isystem", cuda,
           os.path.join(CSRC, "torch_ops.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_ops.cpp:\n{r.stdout}\n{r.stderr}")


def _link_torch_ops(obj: str) -> None:
    tmp = TORCH_OPS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-L", BUILD_DIR, "-lrar", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking _torch_ops.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_OPS_PATH)
    with open(TORCH_OPS_PATH + ".torch", "w") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    torch_obj = os.path.join(BUILD_DIR, "torch_ops.o")
    lacks = binding_lacks()
    if lacks not in (None, "torch"):
        warnings.warn(f"_torch_ops.so is not built (the operators on torch tensors): {lacks} is missing")
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_ops = None if lacks else ex.submit(_compile_torch_ops, torch_obj)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if torch_ops:  # (last: the library does without it)
        torch_ops.result()
        _link_torch_ops(torch_obj)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
