"""In-tree build of libkda.so for sm_103a (nvcc, no cmake) and of the cache calls'
Python binding (the host compiler, against the installed torch).

Each ``csrc/*.cu`` file compiles to an object in parallel, then the objects
link into ``_lib/libkda.so`` against the shared CUDA runtime.  ``csrc/cache_binding.cpp``
becomes ``_lib/_cache_binding.so``, linked to libkda.so beside it.  Rebuilds only
what changed (source or header newer than the object).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libkda.so")
BINDING_PATH = os.path.join(LIB_DIR, "_cache_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the libkda CUDA library cannot be built")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    hs += glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(nvcc: str, src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and os.path.getmtime(obj) >= _headers_mtime()):
        return obj
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, obj)
    return obj


def _compile_binding(src: str) -> str:
    """The binding's object.  It includes torch's headers, the slowest of all to compile:
    -O1, since it computes nothing."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    stamp = obj + ".torch"  # the torch it was built against
    header = os.path.join(INCLUDE, "kda.h")
    if (os.path.exists(obj) and os.path.exists(stamp) and open(stamp).read() == torch.__version__
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), os.path.getmtime(header))):
        return obj
    tmp = obj + f".tmp{os.getpid()}"
    include = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    cmd = [shutil.which("g++") or "c++", "-O1", "-std=c++17", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for i in include for x in ("-isystem", i)], "-c", src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(src)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, obj)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return obj


def _link_binding(obj: str) -> None:
    import torch
    if (os.path.exists(BINDING_PATH) and os.path.getmtime(BINDING_PATH) >= os.path.getmtime(obj)):
        return
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", obj, "-o", tmp, f"-L{LIB_DIR}", "-l:libkda.so",
           f"-L{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda",
           "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _cache_binding.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link libkda.so; return its path."""
    nvcc = _nvcc()
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = list(extra_flags or [])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding, os.path.join(CSRC, "cache_binding.cpp"))
        objs = list(ex.map(lambda s: _compile(nvcc, s, extra), srcs))
        binding_obj = binding.result()
    newest = max(os.path.getmtime(o) for o in objs)
    if os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest:
        _link_binding(binding_obj)
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    libdir = _cuda_lib_dir(nvcc)
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp,
           "-Xlinker", f"-rpath={libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of libkda.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_binding(binding_obj)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
