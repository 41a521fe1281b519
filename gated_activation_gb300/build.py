"""Build the CUDA library ``gated_activation_gb300/_lib/libgated_act.so`` in-tree.

One nvcc per translation unit, run in parallel, then one shared-library link;
beside them one g++ for ``_lib/_training.so``, the training operators' binding
against PyTorch's C++ headers, which links the library.
Target: sm_103a only (``-gencode arch=compute_103a,code=sm_103a``), with
``-lineinfo`` for the profiler and the CUDA runtime linked statically so the
library loads wherever the driver does.  No fast-math: the statistics use
IEEE division and square root.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libgated_act.so")
BINDING = os.path.join(LIB_DIR, "_training.so")
SOURCES = ("api.cu", "gelu_and_mul_sparse.cu", "elementwise.cu",
           "training.cu", "checkpoint.cu", "layer_norm.cu", "balance.cu")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def cflags(extra: list[str] | None = None) -> list[str]:
    return [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", INCLUDE, "-I", CSRC] + (extra or [])


def _compile(src: str, obj: str, extra: list[str]) -> tuple[str, str]:
    cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + cflags(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stderr}")
    return src, r.stderr


def _compile_binding(obj: str) -> None:
    import torch
    headers = os.path.join(os.path.dirname(torch.__file__), "include")
    include = [headers, os.path.join(headers, "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(nvcc()), "..", "include"), INCLUDE]
    cmd = [os.environ.get("CXX", "g++"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj, "-O2",
           "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for p in include:
        cmd += ["-isystem", p]
    _run(cmd, "binding.cpp")


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stderr}")


def _link_binding(obj: str, out: str) -> None:
    import torch
    cmd = [os.environ.get("CXX", "g++"), "-shared", obj, "-o", out, "-L", LIB_DIR, "-lgated_act",
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(os.path.dirname(torch.__file__), "lib")]
    _run(cmd + ["-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_cuda", "-ltorch_cuda"],
         "the binding's link")


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile all sources and link the shared library; returns its path."""
    extra = list(extra or [])
    os.makedirs(LIB_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=LIB_DIR) as tmp:
        objs = [os.path.join(tmp, s.replace(".cu", ".o")) for s in SOURCES]
        binding_obj = os.path.join(tmp, "binding.o")
        with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
            binding = ex.submit(_compile_binding, binding_obj)
            for src, err in ex.map(lambda a: _compile(*a, extra), zip(SOURCES, objs)):
                if verbose and err:
                    print(f"[{src}]\n{err}", file=sys.stderr)
            binding.result()
        out_tmp = os.path.join(tmp, "libgated_act.so")
        _run([nvcc(), "-shared", ARCH, "-cudart", "static", "-o", out_tmp,
              "-Xlinker", "-soname,libgated_act.so"] + objs, "link")
        os.replace(out_tmp, LIB)
        binding_tmp = os.path.join(tmp, "_training.so")
        _link_binding(binding_obj, binding_tmp)
        os.replace(binding_tmp, BINDING)
    return LIB


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return all(os.path.getmtime(p) <= t for p in deps)


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(verbose=v, extra=["-Xptxas", "-v"] if v else None))
