"""Builds libdpg.so, the library's gfx950 shared object, and _binding.so, the
compiled part of the Python binding, in this directory.

hipcc compiles the HIP kernels ahead of time for gfx950 (no JIT) together with
the host planner and the C ABI; the binding is host code against torch's
headers, linked to libdpg.so beside it.  Usage: ``python
deterministic_bf16_projection_amd/build.py`` (run as a file: importing the
package needs the library) or ``build()`` of this module loaded by path.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdpg.so")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("dpg_api.hip", "dpg_grouped.hip", "dpg_route.hip", "dpg_adamw.hip",
                                                   "dpg_norm.hip", "dpg_recurrence.hip", "planner.cpp")]
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "binding.cpp")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
ARCH = "gfx950"

FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-shared",
    # keep the compiler from forming packed-FP32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
]


def _binding_flags():
    import torch
    from torch.utils import cpp_extension
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
             "-D__HIP_PLATFORM_AMD__", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
             "-I", os.path.join(ROOT, "include")]
    rocm = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "include")
    for path in cpp_extension.include_paths() + [sysconfig.get_paths()["include"], rocm]:
        flags += ["-isystem", path]
    for path in cpp_extension.library_paths():
        flags += ["-L" + path]
    return flags + ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-L" + HERE, "-l:libdpg.so",
                    "-Wl,-rpath,$ORIGIN"]


def _compile(cmd, target, verbose):
    tmp = target + ".tmp%d" % os.getpid()
    cmd = cmd + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in res.stdout.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out.strip():
        print(out)
    os.replace(tmp, target)


def build(verbose=False):
    _compile([HIPCC] + FLAGS + SOURCES, LIB, verbose)
    _compile([HIPCC, BINDING_SOURCE] + _binding_flags(), BINDING, verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    print("built", LIB, BINDING)
    sys.exit(0)
