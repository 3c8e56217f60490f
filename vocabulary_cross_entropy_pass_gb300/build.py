"""Build libgbce.so (the CUDA kernels and the C ABI) in-tree with nvcc, and
_gbce_torch.so (torch tensors into that ABI) with g++.

Each translation unit is compiled for sm_103a in its own nvcc process, in
parallel, then linked into vocabulary_cross_entropy_pass_gb300/libgbce.so; the
host module is compiled beside them and linked against it.  The library needs
nvcc alone: it is linked first, and without torch it is all there is to build.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgbce.so")
EXT = os.path.join(HERE, "_gbce_torch.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["ce_api.cu", "ce_aux.cu", "ce_bwd.cu", "ce_fused.cu", "ce_rows.cu", "ce_split.cu",
           "ce_vecrow.cu", "ce_linear.cu", "ce_lmhead.cu", "ce_stream.cu", "ce_stream_geo.cu",
           "ce_vp.cu", "ce_embed.cu", "ce_norm.cu", "ce_logits.cu", "ce_logprobs.cu",
           "ce_softgrad.cu", "ce_distill.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgbce")


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(ROOT, "include", "ce.h"))
    return out


def _torch_dir() -> str | None:
    """The installed torch's folder, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _compile_ext(obj: str) -> None:
    """Compile csrc/ce_torch.cpp against the installed torch's headers."""
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "ce_torch.cpp"), "-o", obj,
           f"-I{inc}", f"-I{inc}/torch/csrc/api/include", f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on ce_torch.cpp:\n{res.stdout}\n{res.stderr}")


def _link_ext(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{HERE}", "-l:libgbce.so", f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
           "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, EXT)


def up_to_date() -> bool:
    made = [LIB, EXT] if _torch_dir() else [LIB]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    ext_obj = os.path.join(BUILD_DIR, "ce_torch.o")
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext, ext_obj) if _torch_dir() else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    res = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcublas"], capture_output=True,
                         text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if ext is not None:
        ext.result()
        _link_ext(ext_obj)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
