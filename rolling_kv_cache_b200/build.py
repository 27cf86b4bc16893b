"""Build the native libraries in place: librc.so with nvcc (sm_100a only), and
_paged.so, the torch extension that hands tensors to its paged operators, with
the host compiler.

Usage: python -m rolling_kv_cache_b200.build [--verbose]
The CUDA runtime is linked statically into librc.so, so the library loads on a
machine without a GPU driver (host-only handles work there; device handles
need a B200).
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "librc.so")
TORCH_SOURCE = os.path.join(CSRC, "paged_torch.cpp")
TORCH_OUT = os.path.join(HERE, "_paged.so")
SOURCES = ["engine.cpp", "api.cu", "rope_kernels.cu", "attn_fwd.cu", "score_kernel.cu", "topc_kernel.cu",
           "rf_kernels.cu",
           "noalloc.cu", "paged_api.cu", "paged_rope.cu", "paged_decode.cu", "paged_attn.cu", "paged_combine.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _newer(out, deps):
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "rc.h"))
    deps.append(os.path.abspath(__file__))
    if not force and _newer(OUT, deps):
        return OUT
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O3", "-shared", "-cudart", "static",
           "-o", OUT + ".tmp"]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += os.environ.get("RC_NVCC_FLAGS", "").split()  # extra -D tuning flags
    cmd += [os.path.join(CSRC, f) for f in SOURCES]
    cmd += ["-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("nvcc failed building librc.so")
    os.replace(OUT + ".tmp", OUT)
    return OUT


def build_torch(verbose: bool = False, force: bool = False) -> str:
    """The torch extension over librc.so (found beside it at load time)."""
    import torch

    header = os.path.join(os.path.dirname(HERE), "include", "rc.h")
    if not force and _newer(TORCH_OUT, [TORCH_SOURCE, header, os.path.abspath(__file__)]):
        return TORCH_OUT
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-o", TORCH_OUT + ".tmp",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-DTORCH_EXTENSION_NAME=_paged"]
    cmd += [f for d in include for f in ("-isystem", d)]
    cmd += [TORCH_SOURCE, "-L" + HERE, "-l:librc.so", "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("the host compiler failed building _paged.so")
    os.replace(TORCH_OUT + ".tmp", TORCH_OUT)
    return TORCH_OUT


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(OUT)
    print(build_torch(verbose="--verbose" in sys.argv, force=True))
