"""Builds libclis.so (CUDA for sm_103a) in-tree with nvcc, and _clis_torch.so, the
torch binding of the calls around a paged cache, with the C++ compiler.

Each translation unit is compiled in parallel to an object file, then linked
into ``certified_fixed_stabilizer_gb300/_lib/libclis.so``.  The CUDA runtime is
linked statically; the driver entry point for tensor maps is resolved at run
time through cudaGetDriverEntryPointByVersion, so no libcuda link is needed.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libclis.so")
TORCH_EXT = os.path.join(OUT_DIR, "_clis_torch.so")
OBJ_DIR = os.path.join(HERE, "_build")

SOURCES = ["clis_api.cu", "certify.cu", "attn_fwd.cu", "attn_bwd.cu", "host_attention.cu", "rope.cu",
           "paged_plan.cu", "paged_decode.cu", "paged_chunk.cu", "paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else (shutil.which("nvcc") or "nvcc")


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _compile_binding() -> str:
    """csrc/binding.cpp against the installed torch's headers."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = os.path.join(OBJ_DIR, "binding.o")
    cmd = [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-w",
           *[f"-I{d}" for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
                                sysconfig.get_paths()["include"])],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling binding.cpp failed:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_EXT + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, f"-L{OUT_DIR}", "-lclis", f"-L{lib}", "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the torch binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_EXT)


def _older(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


HEADER = os.path.join(HERE, "..", "include", "clis.h")


def _stale() -> bool:
    """libclis.so is missing or older than one of its sources."""
    return _older(LIB, [HEADER, *(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp")])


def _torch_tag() -> str:
    """The torch and Python that a binding is built against: it only fits these."""
    import sysconfig

    import torch
    return f"{torch.__version__} abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}"


def _binding_stale() -> bool:
    """_clis_torch.so is missing, older than its source, or built against another torch."""
    if _older(TORCH_EXT, [HEADER, os.path.join(CSRC, "binding.cpp")]):
        return True
    try:
        with open(TORCH_EXT + ".torch") as f:
            return f.read() != _torch_tag()
    except OSError:
        return True


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    """libclis.so, which needs no torch."""
    if not force and not verbose_ptxas and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False) -> str:
    """_clis_torch.so (and libclis.so, which it links)."""
    if force or _binding_stale():
        os.makedirs(OBJ_DIR, exist_ok=True)
        with cf.ThreadPoolExecutor(max_workers=1) as ex:
            obj = ex.submit(_compile_binding)
            build_library(force)
            _link_binding(obj.result())
        with open(TORCH_EXT + ".torch", "w") as f:
            f.write(_torch_tag())
    return TORCH_EXT


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if verbose_ptxas:
        build_library(True, True)
    build_binding(force and not verbose_ptxas)
    return build_library()


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
