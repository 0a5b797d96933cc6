"""Build libfp8fg.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree, and where torch and g++ are there _ffn.so too.

Flags: -O3, no fast-math, no FP contraction (every FMA in the kernels is written explicitly),
packed-FP32 instructions disabled, IEEE fp32 division (HIP's default correctly rounded divide).
"""
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8fg.so")
SOURCES = ["api.hip", "quant.hip", "gemm.hip", "per_tensor.hip", "e5m6.hip", "limited_accum.hip", "act_checkpoint.hip",
           "stream_linear.hip", "moe_few_tokens.hip"]
HOST_SOURCES = ["ffn_api.cpp"]          # argument checks only: no device code
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def flags():
    return ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def host_flags():
    return ["-O2", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def build(verbose: bool = False, extra=()) -> str:
    objs = []
    for src in SOURCES + HOST_SOURCES:
        obj = os.path.join(CSRC, os.path.splitext(src)[0] + ".o")
        dev = [*flags(), *extra] if src in SOURCES else host_flags()
        cmd = [HIPCC, *dev, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
        if r.returncode != 0:
            sys.stderr.write(err + "\n")
            raise RuntimeError(f"hipcc failed on {src}")
        if err.strip() and verbose:
            sys.stderr.write(err + "\n")
        objs.append(obj)
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    # The library must load with every symbol resolved: a kernel missing from the host object (its launch
    # stub not emitted) shows up only here, as an undefined symbol.
    r = subprocess.run([sys.executable, "-c", "import ctypes, sys; ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_LOCAL)",
                        LIB + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr + "\n")
        raise RuntimeError("the built library does not load: " + r.stderr.strip().splitlines()[-1])
    os.replace(LIB + ".tmp", LIB)
    missing = ffn_module_needs()
    if missing:
        # an older binding may not fit the new library; without one, its functions raise at their first call
        if os.path.exists(FFN_MODULE):
            os.remove(FFN_MODULE)
        sys.stderr.write(f"{os.path.basename(FFN_MODULE)}, the Python binding of the feed-forward operators, is not built: "
                         f"it needs {missing}; the C library is complete\n")
    else:
        build_ffn_module(verbose)
    return LIB


FFN_MODULE = os.path.join(HERE, "_ffn.so")


def ffn_module_needs() -> str:
    """What is missing here of what build_ffn_module takes; the C library and its callers take hipcc alone."""
    missing = [] if importlib.util.find_spec("torch") else ["torch"]
    if not shutil.which("g++"):
        missing.append("g++")
    return " and ".join(missing)


def build_ffn_module(verbose: bool = False) -> str:
    """_ffn.so: the compiled Python binding of the feed-forward operators (csrc/ffn_binding.cpp), against the installed
    torch's headers and libraries and libfp8fg.so in this package directory."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cmd = ["g++", "-shared", "-fPIC", "-O2", "-std=c++17", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", os.path.join(base, "include"),
           "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"),
           os.path.join(CSRC, "ffn_binding.cpp"), "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_hip", "-lc10", "-lc10_hip", "-L", HERE, "-lfp8fg", "-Wl,-rpath,$ORIGIN", "-o", FFN_MODULE + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr + "\n")
        raise RuntimeError("g++ failed on csrc/ffn_binding.cpp")
    r = subprocess.run([sys.executable, "-c", "import ctypes, sys, torch; ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_LOCAL)",
                        FFN_MODULE + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr + "\n")
        raise RuntimeError("the built binding does not load: " + r.stderr.strip().splitlines()[-1])
    os.replace(FFN_MODULE + ".tmp", FFN_MODULE)
    return FFN_MODULE


C_CONSUMER = os.path.join(ROOT, "tests", "c_consumer")


def build_c_consumer(verbose: bool = False) -> str:
    """tests/c_consumer: a C++ program that calls the library through include/fp8fg.h only (the GPU test
    tests/test_gpu_c_consumer.py runs it); linked against libfp8fg.so in this package directory."""
    cmd = [HIPCC, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c_consumer.cpp"),
           "-L", HERE, "-lfp8fg", "-Wl,-rpath,$ORIGIN/../fp8_fine_grained_amax_amd", "-o", C_CONSUMER + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stderr + "\n")
        raise RuntimeError("hipcc failed on tests/c_consumer.cpp")
    os.replace(C_CONSUMER + ".tmp", C_CONSUMER)
    return C_CONSUMER


if __name__ == "__main__":
    print(build(verbose=True, extra=sys.argv[1:]))
