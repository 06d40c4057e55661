"""Build libssmscan.so in-tree with nvcc for sm_103a (GB300).

The translation units compile in parallel into ``_build/`` and link into
``selective_state_space_07_gb300/libssmscan.so``. The CUDA runtime is
linked statically, so the library needs only the NVIDIA driver at run time.
Rebuilds happen when any source or header is newer than the library.

Beside it, ``_binding.so``: the short way from Python to some of the calls
(``csrc/binding.cpp``, host code against torch's headers, no kernels). Where
it cannot be built, a warning says so and the ctypes binding makes those calls.
"""
from __future__ import annotations

import glob
import os
import sys
from concurrent.futures import ThreadPoolExecutor
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build", "ssmscan")
LIB = os.path.join(HERE, "libssmscan.so")
SOURCES = ["ssm_fwd.cu", "ssm_bwd.cu", "ssm_api.cu", "ssm_noalloc.cu", "ssm_conv.cu", "ssm_dtproj.cu", "gdn2.cu",
           "mlstm.cu", "glr.cu", "layernorm.cu", "embedding.cu", "w4.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


BINDING = os.path.join(HERE, "_binding.so")
BINDING_TORCH = os.path.join(BUILD, "binding_torch.txt")  # what _binding.so was built for


def _binding_inputs():
    return [os.path.join(CSRC, "binding.cpp"), os.path.abspath(__file__)] + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _binding_tag() -> str:
    """The torch and the Python that run: whose C++ and C interfaces _binding.so uses."""
    import torch
    return f"torch {torch.__version__} {torch._C._GLIBCXX_USE_CXX11_ABI} {sysconfig.get_config_var('SOABI')}"


def binding_fits() -> bool:
    """Whether _binding.so is there and was built for this torch and this Python: only then may it be loaded."""
    try:
        with open(BINDING_TORCH) as f:
            return os.path.exists(BINDING) and f.read() == _binding_tag()
    except OSError:
        return False


def binding_stale() -> bool:
    if not binding_fits():
        return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in _binding_inputs())


def _build_binding() -> None:
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(home, "include"), "-I" + os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), os.path.join(CSRC, "binding.cpp"),
           "-o", tmp, "-L" + os.path.join(home, "lib"), "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-lc10_cuda",
           "-ltorch_cuda", "-Wl,-rpath," + os.path.join(home, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        warnings.warn(f"_binding.so was not built; the ctypes binding makes its calls:\n{r.stdout[-2000:]}\n{r.stderr[-2000:]}")
        return
    if os.path.exists(BINDING_TORCH):
        os.remove(BINDING_TORCH)  # (so that it never speaks of another file than the one that lies there)
    os.replace(tmp, BINDING)
    with open(BINDING_TORCH, "w") as f:
        f.write(_binding_tag())


def _inputs():
    return ([p for p in glob.glob(os.path.join(CSRC, "*")) if not p.endswith("binding.cpp")] + glob.glob(os.path.join(ROOT, "include", "*.h"))
            + [os.path.abspath(__file__)])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and not stale():
        if binding_stale():
            _build_binding()
        return LIB
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding) if force or binding_stale() else None
        results = list(ex.map(compile_one, SOURCES))
        if binding is not None:
            binding.result()
    if verbose or ptxas_info:
        for _, log in results:
            sys.stdout.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
