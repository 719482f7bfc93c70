"""Build libgemm.so (the C-ABI library) in-tree for sm_103a, and the Python
extension ``_quant.so`` that marshals torch tensors into its quantised operators.

Each ``csrc/*.cu`` file is compiled by its own ``nvcc -c`` and ``binding.cpp``
by g++ (in parallel), then linked into
``stage_software_pipelining_gb300/libgemm.so`` against the shared CUDA runtime
and ``_quant.so`` against libgemm.so and torch.  No cmake, one ``-gencode``: a
cold build takes well under a minute, on the x86 dev host (cross-compiling) and
on the Arm GPU host alike.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgemm.so")
BINDING = os.path.join(HERE, "_quant.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    exe = os.path.join(home, "bin", "nvcc")
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found (set CUDA_HOME or put nvcc on PATH)")
    return exe


def cuda_lib_dir() -> str:
    home = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    for sub in ("lib64", "lib", os.path.join("targets", "sbsa-linux", "lib"),
                os.path.join("targets", "x86_64-linux", "lib")):
        d = os.path.join(home, sub)
        if glob.glob(os.path.join(d, "libcudart.so*")):
            return d
    return os.path.join(home, "lib64")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        [os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir() -> str:
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        raise RuntimeError("torch is not installed")
    return os.path.dirname(spec.origin)


def _compile_binding() -> str:
    import sysconfig
    obj = os.path.join(OUT_DIR, "binding.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=1"]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], cuda_inc):
        cmd += ["-isystem", d]
    r = subprocess.run(cmd + ["-c", BINDING_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = os.path.join(_torch_dir(), "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-lgemm", f"-L{libs}", "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}",
           "-Wl,--allow-shlib-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libgemm.so and _quant.so if any source changed; return
    libgemm.so's path.  Where only the extension cannot be built, libgemm.so is
    linked all the same before the error is raised."""
    if not force and not verbose_ptxas and not is_stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    libdir = cuda_lib_dir()
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
           "-Xlinker", f"-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # The library serves C callers where torch's or Python's headers are missing.
    try:
        _link_binding(binding.result())
    except Exception as e:
        raise RuntimeError(f"{LIB} is built, but not the Python extension {BINDING}: {e}") from e
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
