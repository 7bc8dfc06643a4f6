"""Build libqlora_nf4.so in-tree with nvcc for sm_103a (one object per .cu, in parallel), and
_torch_ops.so, the compiled part of the binding (g++ against torch's headers).

Usage: ``python -m bit_nf4_quantized_gb300.build [-v]``.  The results land in
``bit_nf4_quantized_gb300/_build/``; a rebuild happens only when a source or header is newer
than the libraries.
"""

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libqlora_nf4.so")
HOST = os.path.join(CSRC, "host", "torch_ops.cpp")
HOST_LIB = os.path.join(BUILD, "_torch_ops.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files += [os.path.abspath(__file__), HOST]
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(HOST_LIB)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(HOST_LIB))
    return all(os.path.getmtime(f) <= t for f in _deps())


def _cuda_home() -> str:
    return os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"


def _compile_host():
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "torch_ops.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(_cuda_home(), "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, *[a for p in inc for a in ("-isystem", p)], "-c", HOST,
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(HOST)}:\n{r.stdout}\n{r.stderr}")
    return obj, os.path.join(root, "lib")


def _link(cmd, out):
    tmp = out + ".tmp"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every .cu under csrc/ and the compiled binding, and link both; returns the library's path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        host = ex.submit(_compile_host)
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
        host_obj, torch_lib = host.result()
    if verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    _link([nvcc(), *ARCH, "-shared", *[o for o, _ in results]], LIB)
    _link(["g++", "-shared", host_obj, "-L", BUILD, "-lqlora_nf4", "-L", torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"], HOST_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
