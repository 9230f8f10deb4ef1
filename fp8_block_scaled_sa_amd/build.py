"""Builds libdg_fp8.so (the gfx950 HIP library behind include/dg_fp8.h) in-tree,
the host-only binding of some of its calls (_binding.so, against torch's headers),
and the same sources at -O1 -g as libdg_fp8_O1.so: a build with a different
instruction schedule and register allocation, which the tests compare with
the release build bit for bit (a race or a missing wait shows up as a
difference between the two)."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", "library.hip")]
DEPS = SOURCES + [os.path.join(HERE, "csrc", f) for f in (
    "dg_fp8.hip", "kernels.hpp", "quant.hpp", "moe.hpp", "moe_step.hip", "norm.hpp", "gate.hpp", "experts.hpp")
        ] + [os.path.join(ROOT, "include", "dg_fp8.h")]
LIBRARY = os.path.join(HERE, "libdg_fp8.so")
DEBUG_LIBRARY = os.path.join(HERE, "libdg_fp8_O1.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops: keep the compiler from emitting packed fp32 VALU ops.
FLAGS = ["-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I" + os.path.join(ROOT, "include")]


def build(output: str = LIBRARY, extra_flags=()) -> str:
    """Compile every source into one shared library (always recompiles)."""
    tmp = output + ".tmp%d" % os.getpid()
    cmd = [HIPCC, *FLAGS, *extra_flags, *SOURCES, "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, output)
    return output


def build_debug(output: str = DEBUG_LIBRARY) -> str:
    """The same library at -O1 with debug information (-O0 cannot place the
    inline-asm LDS-DMA operands in scalar registers)."""
    tmp = output + ".tmp%d" % os.getpid()
    flags = ["-O1", "-g"] + [f for f in FLAGS if f != "-O3"]
    subprocess.check_call([HIPCC, *flags, *SOURCES, "-o", tmp])
    os.replace(tmp, output)
    return output


def build_binding(output: str = BINDING) -> str:
    """Compile the host-only binding against the installed torch."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    tmp = output + ".tmp%d" % os.getpid()
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = ["-I" + p for p in [os.path.join(ROOT, "include"), *include_paths(), sysconfig.get_path("include")]]
    subprocess.check_call([CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", *includes,
                           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, BINDING_SOURCE, "-o", tmp,
                           "-L" + torch_lib, "-lc10", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, output)
    return output


def is_stale(output: str = LIBRARY) -> bool:
    if not os.path.exists(output):
        return True
    t = os.path.getmtime(output)
    return any(os.path.getmtime(d) > t for d in DEPS)


if __name__ == "__main__":
    print(build())
    print(build_debug())
    print(build_binding())
