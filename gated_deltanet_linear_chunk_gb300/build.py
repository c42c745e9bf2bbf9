"""Builds the CUDA library (libgdn) in-tree for sm_103a with nvcc.

Each .cu under csrc/ compiles to an object in parallel; the objects link into
one shared library with the CUDA runtime linked statically, so the library
loads on a machine without a GPU (only the C ABI symbols are exported).  A
second variant, libgdn_debug, is built with GDN_DEBUG: the same kernels plus
device-side checks of the inputs' preconditions and of the kernels' indices.
The host compiler builds the extension module that marshals the block
operators' tensors.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-Xptxas", "-warn-spills", "--expt-relaxed-constexpr"]


def library_path(debug: bool = False) -> str:
    """The release library, or with `debug` the GDN_DEBUG one (device-side
    checks of the inputs' preconditions and of the kernels' indices)."""
    name = "libgdn_debug" if debug else "libgdn"
    return os.path.join(BUILD, f"{name}_{platform.machine()}.so")


def binding_path() -> str:
    """The extension module that marshals the block operators' tensors, for this
    Python and PyTorch: it uses their C++ interfaces, which others do not share."""
    import torch
    return os.path.join(BUILD, f"gdn_block_binding_{platform.machine()}_"
                               f"{sysconfig.get_config_var('SOABI')}_torch-{torch.__version__}.so")


def _binding_command(out: str):
    """Compiles csrc/block_binding.cpp against this Python and PyTorch; their
    libraries are those that `import torch` has already loaded."""
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", os.path.join(home, "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(cuda, "include"), "-I", INCLUDE,
            os.path.join(CSRC, "block_binding.cpp"), "-o", out,
            "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
            "-lc10", "-lc10_cuda"]


def _build_binding(force: bool) -> None:
    out = binding_path()
    if not (force or _stale(out)):
        return
    os.makedirs(BUILD, exist_ok=True)
    tmp = out + ".tmp"
    r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on block_binding.cpp:\n{r.stderr}")
    os.replace(tmp, out)


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    newest = max(os.path.getmtime(p) for p in _deps())
    return os.path.getmtime(out) < newest


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug=None) -> str:
    """Compile every CUDA source and link the library: debug=None builds the
    release and the GDN_DEBUG variants and the binding (their sources compiled
    in one parallel pool), False the release variant and the binding, True the
    GDN_DEBUG one.  The libraries need nvcc alone: they are linked also where
    the binding cannot be compiled (g++, Python's and PyTorch's headers), which
    is raised after.  Returns the path of the
    release library (or of the one variant asked for)."""
    variants = [False, True] if debug is None else [bool(debug)]
    todo = [v for v in variants if force or _stale(library_path(v))]
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_build_binding, force) if debug is not True else None
        _build_libraries(todo, verbose, extra_flags)
    if binding:
        binding.result()
    return library_path(False if debug is None else bool(debug))


def _build_libraries(todo, verbose: bool, extra_flags) -> None:
    """Compiles and links the variants of the library in `todo`."""
    if todo:
        nvcc = _nvcc()
        srcs = _sources()

        def obj_dir(dbg):
            return os.path.join(BUILD, "debug") if dbg else BUILD

        def compile_one(job):
            dbg, src = job
            obj = os.path.join(obj_dir(dbg), os.path.basename(src) + f".{platform.machine()}.o")
            flags = [*NVCC_FLAGS, *extra_flags] + (["-DGDN_DEBUG"] if dbg else [])
            cmd = [nvcc, *ARCH, *flags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
            if verbose and r.stderr:
                print(r.stderr)
            return obj

        for dbg in todo:
            os.makedirs(obj_dir(dbg), exist_ok=True)
        jobs = [(dbg, src) for dbg in todo for src in srcs]
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            objs = list(ex.map(compile_one, jobs))
        for dbg in todo:
            out = library_path(dbg)
            mine = [o for (d, _), o in zip(jobs, objs) if d == dbg]
            tmp = out + ".tmp"
            cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-Xcompiler", "-fPIC", *mine,
                   "-o", tmp]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
