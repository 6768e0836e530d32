"""Build in-tree: libkvpack.so (the sm_100a kernels and their C ABI) with nvcc, and _call.so (the native part of
the Python binding) with the C++ compiler against torch's headers."""
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvpack.so")
CALL = os.path.join(HERE, "_call.so")
CALL_FOR = CALL + ".for"            # the torch and Python that _call.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    out = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            out.append(os.path.join(CSRC, f))
    out.append(os.path.join(ROOT, "include", "kvpack.h"))
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(s) for s in sources())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    cmd = [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
           "-Xcompiler", "-fPIC,-O2", "-shared", "-I", os.path.join(ROOT, "include"),
           "-o", LIB + ".tmp", os.path.join(CSRC, "kvpack.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def _torch():
    """torch's folder and version, without importing it."""
    at = importlib.util.find_spec("torch").submodule_search_locations[0]
    return at, runpy.run_path(os.path.join(at, "version.py"))["__version__"]


def call_for() -> str:
    return f"torch {_torch()[1]}, {sysconfig.get_config_var('SOABI')}"


def call_is_fresh() -> bool:
    """Whether _call.so is newer than its sources and was built for this torch and Python."""
    src = [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "kvpack.h")]
    if not os.path.exists(CALL) or not os.path.exists(CALL_FOR):
        return False
    with open(CALL_FOR) as f:
        return f.read() == call_for() and os.path.getmtime(CALL) >= max(os.path.getmtime(s) for s in src)


def build_call(force: bool = False) -> str:
    """The binding's extension; it links to libkvpack.so next to it."""
    if not force and call_is_fresh():
        return CALL
    torch, version = _torch()
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-w", *(f"-I{i}" for i in inc),
           f'-DKVPACK_TORCH="{version}"', "-o", CALL + ".tmp", os.path.join(CSRC, "binding.cpp"), f"-L{HERE}",
           "-l:libkvpack.so", f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    subprocess.check_call(cmd)
    if os.path.exists(CALL_FOR):
        os.remove(CALL_FOR)             # until the new pair is complete
    os.replace(CALL + ".tmp", CALL)
    with open(CALL_FOR, "w") as f:
        f.write(call_for())
    return CALL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_call(force="--force" in sys.argv))
