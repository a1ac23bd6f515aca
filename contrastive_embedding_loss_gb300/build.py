"""Build the CUDA library in-tree: ``contrastive_embedding_loss_gb300/_build/libuf_contrastive.so``.

nvcc compiles each translation unit for sm_103a only (in parallel), then links one
shared object with the CUDA runtime linked statically, so loading the library needs no
GPU and no libcuda (the driver entry point is resolved at the first call).  The library needs
nvcc alone.  Where torch for CUDA is installed, g++ builds ``_layers_native-<torch's version>.so`` beside
it, the Python module that calls the library with torch tensors: one that was built against
another torch is not found, rather than loaded.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB_NAME = "libuf_contrastive.so"
SOURCES = ["wgt_kernel.cu", "gemm_kernel.cu", "fwd_kernel.cu", "aux_kernels.cu", "uf_contrastive.cu", "uf_static.cu",
           "dense_kernel.cu", "skinny_kernel.cu", "norm_kernels.cu", "act_kernels.cu", "adamw_kernel.cu", "uf_layers.cu"]
NATIVE_NAME = "_layers_native"
NATIVE_SOURCE = "layers_binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _digest(*more: str) -> str:
    h = hashlib.sha1()
    for d in (CSRC, INCLUDE):
        for f in sorted(os.listdir(d)):
            with open(os.path.join(d, f), "rb") as fh:
                h.update(f.encode() + fh.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    h.update(os.uname().machine.encode())
    h.update(" ".join(more).encode())
    return h.hexdigest()[:16]


def _fresh(out: str, digest: str) -> bool:
    """Whether ``out`` was built from what ``digest`` stands for."""
    stamp = out + ".stamp"
    return os.path.exists(out) and os.path.exists(stamp) and open(stamp).read() == digest


def _stamp(out: str, digest: str) -> None:
    with open(out + ".stamp", "w") as f:
        f.write(digest)


def lib_path() -> str:
    return os.path.join(BUILD, LIB_NAME)


def torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "none"


def native_path() -> str:
    return os.path.join(BUILD, f"{NATIVE_NAME}-{torch_version()}.so")


def _build_native(force: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None or not os.path.exists(os.path.join(os.path.dirname(spec.origin), "lib", "libc10_cuda.so")):
        return
    out = native_path()
    digest = _digest(torch_version())
    if not force and _fresh(out, digest):
        return
    torch_dir = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = out + f".tmp{os.getpid()}"
    include = [f"{torch_dir}/include", f"{torch_dir}/include/torch/csrc/api/include", f"{cuda}/include",
               sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", *[f"-I{d}" for d in include],
           os.path.join(CSRC, NATIVE_SOURCE), "-o", tmp, f"-L{torch_dir}/lib", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda", f"-Wl,-rpath,{torch_dir}/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {NATIVE_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    _stamp(out, digest)


def _build_library(force: bool, verbose: bool) -> None:
    out, digest = lib_path(), _digest()
    if not force and _fresh(out, digest):
        return
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [exe, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = out + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    _stamp(out, digest)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is not up to date and return the path of the shared library."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        native = ex.submit(_build_native, force)
        _build_library(force, verbose)
        native.result()
    return lib_path()


if __name__ == "__main__":
    print(build(force=True, verbose=True))
