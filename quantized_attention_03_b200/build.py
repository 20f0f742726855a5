"""Build ``libsage.so`` (the C-ABI CUDA library) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libsage.so")
BINDING = os.path.join(HERE, "_binding.so")     # tensors to C ABI calls (csrc/binding.cpp)
SOURCES = ["api.cu", "kv4_api.cu", "quant.cu", "attn_sm100.cu", "decode.cu", "rope.cu", "kv4.cu",
           "kv4_attn.cu", "selftest.cu"]
HEADERS = ["sage_common.cuh", "sm100_ptx.cuh", "quant_codes.cuh", "decode.cuh", "rope.cuh",
           "kv4.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def binding_for() -> str:
    """What a binding fits: the Python and the torch that it is compiled against."""
    import sysconfig

    import torch
    return (f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__} "
            f"cxx11abi {int(torch.compiled_with_cxx11_abi())}")


def _binding_stale() -> bool:
    deps = [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "sage.h")]
    if not os.path.exists(BINDING) or any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in deps):
        return True
    try:
        with open(BINDING + ".for") as f:
            return f.read() != binding_for()
    except OSError:
        return True


def build_binding(force: bool = False) -> str:
    """Compile the Python extension that makes the rotary and 4-bit cache calls (g++, torch's
    headers and libraries)."""
    if not force and not _binding_stale():
        return BINDING
    import sysconfig

    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(base, "include"), os.path.join(base, "include/torch/csrc/api/include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(base, "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DBUILT_FOR="{binding_for()}"',
           *(x for p in include for x in ("-isystem", p)), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(binding_for())
    return BINDING


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "sage.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library, and the Python extension beside it. The library takes nvcc alone; where
    the extension cannot be compiled (no torch, no Python headers), that is a warning, and the
    calls that go through it raise."""
    build_library(force, verbose)
    try:
        build_binding(force)
    except (ImportError, OSError, RuntimeError) as e:
        if not isinstance(e, ImportError) and os.path.exists(BINDING):
            os.remove(BINDING)                         # an older one, which may not fit the library
        warnings.warn(f"no Python extension for the rotary and 4-bit cache calls: {e}")
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source into one shared library (objects built in parallel)."""
    if not force and not _stale():
        return LIB
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [_nvcc(), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(f"--- {src}\n{text}")
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(f"--- {s}\n{t}" for s, t in failed))
    tmp = LIB + ".tmp"
    subprocess.run([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                    "-Xcompiler", "-fPIC", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
