"""Compile the CUDA library ``libkda.so`` in-tree for sm_103a, and the compiled
part of the Python binding, ``_binding.so``.

All translation units in one nvcc call (compiled side by side), one ``-gencode`` (compute_103a /
sm_103a), the CUDA runtime linked statically so the library only needs the
driver at run time.  The binding's part is host code against PyTorch's headers,
for one version of PyTorch and Python, which is noted beside it; where it cannot
be built, none is left behind and ``api.py`` does its work.
"""

from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, f)
           for f in ("kda_kernels.cu", "kda_conv.cu", "kda_blocks.cu", "kda_append.cu",
                     "kda_attend.cu", "kda_logprobs.cu", "kda_decode.cu",
                     "kda_prefill.cu")]
DEPENDS = SOURCES + [
    os.path.join(CSRC, "kda_device.cuh"),
    os.path.join(CSRC, "kda_async.cuh"),
    os.path.join(CSRC, "kda_align.cuh"),
    os.path.join(CSRC, "kda_tc.cuh"),
    os.path.join(CSRC, "kda_cache.cuh"),
    os.path.join(CSRC, "kda_delta.cuh"),
    os.path.join(ROOT, "include", "kda.h"),
]
LIBRARY = os.path.join(PKG, "libkda.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc")
    if cand:
        return cand
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(cuda_home, "bin", "nvcc")


def _older(output: str, sources) -> bool:
    if not os.path.exists(output):
        return True
    built = os.path.getmtime(output)
    return any(os.path.getmtime(src) > built for src in sources)


def _stale() -> bool:
    return _older(LIBRARY, DEPENDS)


def compile_command(output: str, extra=(), sources=None) -> list[str]:
    return [
        nvcc_path(),
        *ARCH_FLAGS,
        "-O3",
        "-lineinfo",
        "-std=c++17",
        "--threads",
        "0",
        "-shared",
        "-Xcompiler",
        "-fPIC",
        "-cudart",
        "static",
        "-I",
        os.path.join(ROOT, "include"),
        *extra,
        "-o",
        output,
        *(SOURCES if sources is None else sources),
    ]


def _built_for() -> str:
    """What a build of the binding's part is for ("" where PyTorch is missing)."""
    try:
        import torch
    except ImportError:
        return ""
    return f"PyTorch {torch.__version__}, Python {platform.python_version()}"


def _binding_stale() -> bool:
    if _older(BINDING, [BINDING_SOURCE, os.path.join(ROOT, "include", "kda.h")]):
        return True
    try:
        with open(BINDING + ".for") as f:
            return f.read() != _built_for()
    except OSError:
        return True


def binding_command(output: str) -> list[str]:
    import torch

    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    home = os.path.dirname(torch.__file__)
    headers = os.path.join(home, "include")
    return [
        "g++", "-std=c++17", "-O2", "-fPIC", "-shared",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        f'-DKDA_TORCH_VERSION="{torch.__version__}"',
        "-I", os.path.join(ROOT, "include"),
        "-I", sysconfig.get_paths()["include"],
        "-I", headers,
        "-I", os.path.join(headers, "torch", "csrc", "api", "include"),
        "-I", os.path.join(cuda, "include"),
        "-o", output, BINDING_SOURCE,
        "-L", os.path.join(home, "lib"),
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
    ]


def _build_library(verbose: bool) -> None:
    tmp = LIBRARY + f".tmp{os.getpid()}"
    extra = ["-Xptxas", "-v"] if verbose else []
    subprocess.run(compile_command(tmp, extra), check=True)
    os.replace(tmp, LIBRARY)


def _build_binding() -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    try:
        subprocess.run(binding_command(tmp), check=True, capture_output=True, text=True)
    except (ImportError, OSError, subprocess.SubprocessError) as error:
        # an old one would be given the argument structures of another kda.h
        for path in (BINDING, BINDING + ".for", tmp):
            if os.path.exists(path):
                os.remove(path)
        print("the compiled part of the binding was not built; api.py does its work:\n"
              f"{error}\n{(getattr(error, 'stderr', None) or '')[:2000]}", file=sys.stderr)
        return
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(_built_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``libkda.so`` and ``_binding.so``, side by side, where a source is
    newer (for the binding: or PyTorch another); return the library's path."""
    with ThreadPoolExecutor(2) as pool:
        jobs = []
        if force or _binding_stale():
            jobs.append(pool.submit(_build_binding))
        if force or _stale():
            jobs.append(pool.submit(_build_library, verbose))
        for job in jobs:
            job.result()
    return LIBRARY


VARIANT_DIR = os.path.join(PKG, "_variants")


def build_variant(name: str, defines, force: bool = False) -> str:
    """Build a test variant of the library with extra preprocessor
    definitions, into _variants/libkda_<name>.so; never the product library.
    The tests use it for paths no input of the C ABI can reach (a wait that
    runs out)."""
    os.makedirs(VARIANT_DIR, exist_ok=True)
    out = os.path.join(VARIANT_DIR, f"libkda_{name}.so")
    if not force and os.path.exists(out) and not _stale_against(out):
        return out
    tmp = out + f".tmp{os.getpid()}"
    extra = [f"-D{d}" for d in defines]
    subprocess.run(compile_command(tmp, extra), check=True)
    os.replace(tmp, out)
    return out


def _stale_against(path: str) -> bool:
    built = os.path.getmtime(path)
    return any(os.path.getmtime(src) > built for src in DEPENDS)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
