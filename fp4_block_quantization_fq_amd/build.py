"""Build libfq.so (the HIP kernels and the C ABI) for gfx950, and the Python
extension _fq_binding.so over it, in-tree.

hipcc cross-compiles here without a GPU.  Flags that the numerics rely on:
  -ffp-contract=off                no silent a*b+c fusion: each float operation
                                   in the quantizers is the one written
  -fhip-fp32-correctly-rounded-divide-sqrt
                                   '/' on float is IEEE correctly rounded
  -fno-gpu-flush-denormals-to-zero FP32 subnormals are kept
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                   no packed-FP32 VALU instructions
"""
import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfq.so")
BINDING = os.path.join(PKG, "_fq_binding.so")

SOURCES = ["fq_api.cpp", "fq_kernels.hip", "fq_gemm.hip", "fq_hadamard.hip", "fq_outcontrol.hip",
           "fq_norm.hip", "fq_moe.hip", "fq_adamw.hip"]
ARCH = "gfx950"

COMMON = [
    "-std=c++17", "-O3", "-fPIC", f"--offload-arch={ARCH}",
    "-ffp-contract=off", "-fno-fast-math",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _hipcc() -> str:
    for c in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.isabs(c) and os.path.exists(c):
            return c
    return "hipcc"


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
    if verbose and msg.strip():
        print(msg, flush=True)
    return obj


def _compile_binding(verbose: bool) -> str:
    """Host code only: torch's headers read the tensors, the C ABI is linked."""
    import sysconfig

    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "fq_binding.o")
    dirs = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", "-c", os.path.join(CSRC, "fq_binding.cpp"),
           *[f"-isystem{d}" for d in dirs], "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fq_binding.cpp:\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, flush=True)
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    from torch.utils import cpp_extension
    cmd = ["g++", "-shared", obj, "-o", BINDING + ".tmp", f"-L{PKG}", "-l:libfq.so",
           "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in cpp_extension.library_paths()],
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_compile_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    # --no-undefined: a symbol missing from the sources fails here, not at load time
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,--no-undefined", *objs,
           "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    _link_binding(binding.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
