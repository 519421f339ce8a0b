"""Build the CUDA library in-tree: dense_tensor_core_gb300/libdtc_gemm.so (sm_103a only), and the
native part of the Python binding, dense_tensor_core_gb300/_ffn_native.so.

One translation unit per kernel family plus the API unit, compiled in parallel with nvcc (one
-gencode), then linked into one shared library. The CUDA runtime is linked statically so the
library loads without a GPU (the CPU tests check its exports) and carries no rpath. The library needs
neither torch nor Python's headers. The binding module is host code against torch's headers, compiled
beside the kernels (about 10 s) and linked against the library in its own folder; where torch is not
installed it is left out, and where it does not compile the library is in place all the same.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdtc_gemm.so")
NATIVE = os.path.join(HERE, "_ffn_native.so")
OBJ_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cand, "bin", "nvcc")
    return p if os.path.exists(p) else (shutil.which("nvcc") or "nvcc")


def _headers(folder, *kinds):
    return [os.path.join(folder, f) for f in os.listdir(folder) if f.endswith(kinds)]


def _due(target, inputs):
    """Whether `target` is missing or older than one of its inputs."""
    return not os.path.exists(target) or os.path.getmtime(target) < max(map(os.path.getmtime, inputs))


def _native_sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cpp"))


def _compile_native(obj_dir):
    """The binding module's objects (no GPU code; torch's own headers and ABI), compiled side by side."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            cuda, sysconfig.get_paths()["include"], INCLUDE]
    flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
    flags += [x for d in dirs for x in ("-isystem" if "torch" in d else "-I", d)]

    def one(src):
        obj = os.path.join(obj_dir, os.path.basename(src)[:-4] + ".o")
        subprocess.check_call([shutil.which("g++") or "g++", *flags, "-c", src, "-o", obj])
        return obj

    srcs = _native_sources()
    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        return list(ex.map(one, srcs))


def _link_native(objs, tmp):
    import torch

    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.check_call(
        [shutil.which("g++") or "g++", "-shared", *objs, "-o", tmp, "-L" + HERE, "-ldtc_gemm",
         "-Wl,-rpath,$ORIGIN", "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
         "-lc10_cuda"])


def _compile(src, obj_dir, verbose_ptxas):
    obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
           "-I", CSRC, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.check_call(cmd)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    srcs = sources()
    headers = _headers(INCLUDE, ".h")
    library = force or _due(LIB, srcs + headers + _headers(CSRC, ".cuh", ".h"))
    native = importlib.util.find_spec("torch") is not None and (
        force or _due(NATIVE, headers + _native_sources() + [os.path.join(CSRC, "binding.h")]))
    if not library and not native:
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    # objects in a directory of this build's own, so concurrent builds cannot mix their files
    with tempfile.TemporaryDirectory(dir=OBJ_DIR) as obj_dir, \
            ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_native, obj_dir) if native else None
        if library:
            objs = list(ex.map(lambda s: _compile(s, obj_dir, verbose_ptxas), srcs))
            tmp = LIB + ".tmp%d" % os.getpid()
            subprocess.check_call([nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
            os.replace(tmp, LIB)
        if native:
            tmp = NATIVE + ".tmp%d" % os.getpid()
            _link_native(binding.result(), tmp)
            os.replace(tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
