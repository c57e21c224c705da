"""Builds the in-tree CUDA library ``libkda_gb300.so`` for sm_103a with nvcc.

Each translation unit under ``csrc/`` compiles in its own nvcc process (in
parallel), then one link step produces the shared library next to this file in
``_build/``. Only ``-gencode arch=compute_103a,code=sm_103a`` is emitted.

``csrc/binding.cpp``, the compiled part of the Python binding, becomes
``_build/kda_gb300_binding.so``, linked against that library and torch's headers. Where g++ or the Python
or torch headers are missing, the library is built without it: the calls that need it raise then.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libkda_gb300.so")
BINDING_PATH = os.path.join(BUILD_DIR, "kda_gb300_binding.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "kda.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(made: str, files) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in files)


def up_to_date(lib_path: str = LIB_PATH) -> bool:
    return _newer(lib_path, _deps())


def binding_up_to_date() -> bool:
    return _newer(BINDING_PATH, [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)])


def _compile_binding():
    """Compiles csrc/binding.cpp; returns its object and what links it."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj, ["-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _link(cmd, path):
    tmp = path + f".{os.getpid()}.tmp"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str = LIB_PATH) -> str:
    """Compile every ``csrc/*.cu`` and link ``_build/libkda_gb300.so``; returns its path.

    ``extra_flags`` and another ``lib_path`` build a variant of the library in its own folder
    beside it (the failure-detection test builds one with a short wait limit that way)."""
    with_binding = lib_path == LIB_PATH and (force or not binding_up_to_date())
    with_library = force or not up_to_date(lib_path)
    if not with_binding and not with_library:
        return lib_path
    build_dir = os.path.dirname(lib_path)
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources() if with_library else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_compile_binding) if with_binding else None
        objs = list(ex.map(compile_one, srcs))
    if with_library:
        _link([nvcc, *ARCH, "-shared", *objs, "-cudart", "static"], lib_path)
    if with_binding:
        try:
            obj, libs = binding.result()
            _link(["g++", "-shared", obj, "-L", build_dir, "-l:" + os.path.basename(lib_path), "-Wl,-rpath,$ORIGIN", *libs],
                  BINDING_PATH)
        except (ImportError, OSError, RuntimeError) as e:
            if os.path.exists(BINDING_PATH):  # of other sources
                os.remove(BINDING_PATH)
            warnings.warn(f"the compiled part of the Python binding is missing, and the calls that need it will raise: {e}")
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=(["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])))
