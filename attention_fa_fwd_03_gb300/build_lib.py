"""Compile the CUDA library ``libfa_gb300.so`` in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process (in parallel), then
the objects are linked into one shared library next to this file. The CUDA
runtime is linked statically, so loading the library needs no CUDA driver
until the first call that touches the GPU.

Beside it ``_paged.so`` is built, the Python binding of the paged-cache calls
and of differentiable attention (csrc/paged_binding.cpp), by the host compiler
against the headers of the PyTorch that is installed, and again when that is
another one.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa_gb300.so")
BINDING_SRC = os.path.join(CSRC, "paged_binding.cpp")
BINDING_DEPS = [BINDING_SRC, os.path.join(CSRC, "autograd_binding.h")]
BINDING = os.path.join(HERE, "_paged.so")
BINDING_FOR = os.path.join(BUILD, "paged_binding.pytorch")  # what it was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xptxas", "-v", "--expt-relaxed-constexpr"] + ARCH


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def _library_current() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _pytorch() -> str | None:
    """Which PyTorch the binding would be built against (its version, place and date, and the Python's), without importing it;
    None where there is none."""
    import importlib.metadata
    import importlib.util
    try:
        spec = importlib.util.find_spec("torch")
        if spec is None or not spec.origin:
            return None
        version = importlib.metadata.version("torch")
        installed = int(os.path.getmtime(spec.origin))
    except (ImportError, ValueError, OSError):
        return None
    return f"{version} {os.path.dirname(spec.origin)} {installed} {sys.implementation.cache_tag}"


def _binding_current(pytorch: str) -> bool:
    if not _newer(BINDING, BINDING_DEPS + [os.path.abspath(__file__)]
                  + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return False
    try:
        with open(BINDING_FOR) as fh:
            return fh.read() == pytorch
    except OSError:
        return False


def up_to_date() -> bool:
    """Whether build() has nothing to do: the library is newer than its sources, and so is the binding, which was built
    against the PyTorch that is there now."""
    pytorch = _pytorch()
    return _library_current() and (pytorch is None or _binding_current(pytorch))


def _binding_flags() -> tuple[list[str], list[str]]:
    """Compiler flags and link flags of the Python binding."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    abi = int(torch.compiled_with_cxx11_abi())
    lib = os.path.join(root, "lib")
    return (["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *(f"-I{d}" for d in inc)],
            [f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}",
             f"-L{HERE}", "-l:libfa_gb300.so", "-Wl,-rpath,$ORIGIN"])


def build(force: bool = False, verbose: bool = False) -> str:
    """Build the library, and the Python binding of the paged calls, where a source is newer or the binding was built
    against another PyTorch; return the library's path. Without PyTorch the library alone is built."""
    pytorch = _pytorch()
    library = force or not _library_current()
    binding = pytorch is not None and (force or not _binding_current(pytorch))
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    binding_obj = os.path.join(BUILD, "paged_binding.o")
    cflags, ldflags = _binding_flags() if binding else ([], [])
    nvcc = _nvcc()
    cmds = []
    if library:
        for src in sources():
            obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
            cmds.append((src, obj + ".log", [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]))
    if binding:
        cmds.append((BINDING_SRC, binding_obj + ".log", ["g++", *cflags, "-c", BINDING_SRC, "-o", binding_obj]))
    procs = []
    for src, log, cmd in cmds:
        fh = open(log, "w")
        procs.append((src, log, fh, subprocess.Popen(cmd, stdout=fh, stderr=subprocess.STDOUT)))
    failed = []
    for src, log, fh, p in procs:
        p.wait()
        fh.close()
        if p.returncode != 0:
            failed.append((src, log))
        elif verbose:
            sys.stdout.write(open(log).read())
    if failed:
        msgs = []
        for src, log in failed:
            msgs.append(f"--- {os.path.basename(src)} ---\n" + open(log).read()[-6000:])
        raise RuntimeError("compilation failed:\n" + "\n".join(msgs))
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in sources()]
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if binding:
        tmp = BINDING + f".tmp{os.getpid()}"
        subprocess.run(["g++", "-shared", "-o", tmp, binding_obj, *ldflags], check=True)
        os.replace(tmp, BINDING)
        with open(BINDING_FOR, "w") as fh:
            fh.write(pytorch)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
