"""Builds libdsa_b200.so in-tree for sm_100a with nvcc, and with the host compiler the Python
binding _binding.so of the paged calls over it (no JIT)."""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdsa_b200.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    hdr = os.path.join(os.path.dirname(HERE), "include", "dsa.h")
    return any(os.path.getmtime(s) > t for s in sources() + [hdr])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Builds the library and its Python binding where a source is newer; returns the library's path."""
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "nvcc")
        cmd = [nvcc, "-O3", "-std=c++17", *ARCH, "-lineinfo", "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
               "-cudart", "static", "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills",
               *extra, "-o", LIB + ".tmp", os.path.join(CSRC, "libdsa.cu")]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    build_binding(force, verbose)
    return LIB


def _binding_stamp() -> str:
    """What the binding holds of the interpreter and the torch that it was built against."""
    import torch
    return f"dsa-binding python {sysconfig.get_python_version()} torch {torch.__version__}"


def needs_binding() -> bool:
    hdr = os.path.join(os.path.dirname(HERE), "include", "dsa.h")
    if not os.path.exists(BINDING) or any(os.path.getmtime(f) > os.path.getmtime(BINDING) for f in (BINDING_SRC, hdr)):
        return True
    with open(BINDING, "rb") as f:  # torch's C++ interface changes with its version
        return _binding_stamp().encode() + b"\0" not in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The native marshalling of the paged calls: a Python module on torch's headers that calls the
    C ABI of libdsa_b200.so beside it."""
    if not force and not needs_binding():
        return BINDING
    import torch
    tdir = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DDSA_BINDING_STAMP="{_binding_stamp()}"',
           "-I" + os.path.join(tdir, "include"), "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
           BINDING_SRC, "-o", BINDING + ".tmp", "-L" + os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", "-L" + HERE,
           "-l:libdsa_b200.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
