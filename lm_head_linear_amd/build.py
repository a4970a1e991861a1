"""Build liblce.so (HIP for gfx950) in-tree with hipcc.

Every .hip / .cpp source under csrc/ and csrc_ops/ is compiled for gfx950 only and linked
into lm_head_linear_amd/liblce.so.  Packed-fp32 instructions are disabled
for all device code.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "liblce.so")
BINDING = os.path.join(HERE, "_lce_torch.so")     # torch tensors -> liblce.so
OBJ_DIR = os.path.join(HERE, "_build")

# csrc/ holds the losses, csrc_ops/ the operators that stand next to them.
SOURCES = ["csrc/lce_contract.cpp", "csrc/lce_ce.hip", "csrc/lce_distill.hip",
           "csrc_ops/beam.hip", "csrc_ops/checkpoint.hip", "csrc_ops/linear.hip"]

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
ARCH = os.environ.get("LCE_OFFLOAD_ARCH", "gfx950")

COMMON = ["-O3", "-fPIC", "-std=c++17", f"-I{INCLUDE}", "-Wall", "-Wno-unused-function"]
DEVICE = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-munsafe-fp-atomics"]


def _compile(src: str) -> str:
    path = os.path.join(HERE, src)
    obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
    if src.endswith(".hip"):
        cmd = [HIPCC, "-x", "hip", *DEVICE, *COMMON, "-c", path, "-o", obj]
    else:
        cmd = [HIPCC, *COMMON, "-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"compile failed: {src}")
    return obj


def _compile_binding() -> str:
    """Compile the torch binding (host code only)."""
    import sysconfig

    from torch.utils import cpp_extension

    obj = os.path.join(OBJ_DIR, "torch_binding.cpp.o")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    includes = [INCLUDE, *cpp_extension.include_paths(), os.path.join(rocm, "include"),
                sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-DTORCH_EXTENSION_NAME=_lce_torch", *[f"-I{i}" for i in includes], "-c",
           os.path.join(HERE, "csrc_ops", "torch_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("compile failed: torch_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension

    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", "-Wl,-rpath,$ORIGIN", "-o", tmp, obj, f"-L{HERE}", "-l:liblce.so",
           *[f"-L{d}" for d in cpp_extension.library_paths()], "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed: _lce_torch.so")
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    # -z defs: an unresolved symbol (e.g. a kernel stub the host pass dropped)
    # fails the link instead of the first dlopen.
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-z,defs", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
