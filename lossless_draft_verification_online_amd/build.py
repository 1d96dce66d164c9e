"""Builds libsdv.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", "sdv.hip"), os.path.join(PKG, "csrc", "commit.hip"),
           os.path.join(PKG, "csrc", "sample.hip"), os.path.join(PKG, "csrc", "cache.hip"),
           os.path.join(PKG, "csrc", "attend.hip"), os.path.join(PKG, "csrc", "cache8.hip"),
           os.path.join(PKG, "csrc", "attend8.hip"), os.path.join(PKG, "csrc", "pages.hip"),
           os.path.join(PKG, "csrc", "sdcp_uniforms.cpp")]
DEPENDS = SOURCES + [os.path.join(PKG, "csrc", "sdv_device.hpp"), os.path.join(PKG, "csrc", "split.hpp"),
                     os.path.join(PKG, "csrc", "cache_view.hpp"), os.path.join(PKG, "csrc", "attend_unit.hpp"),
                     os.path.join(PKG, "csrc", "attend_rows.hpp"),
                     os.path.join(PKG, "csrc", "cache8_view.hpp"), os.path.join(PKG, "csrc", "launch.hpp"),
                     os.path.join(ROOT, "include", "sdv.h")]
LIBRARY = os.path.join(PKG, "libsdv.so")
# The Python module that marshals the newer calls' tensors: host code, on torch's C++ interface.
MARSHAL_SOURCE = os.path.join(PKG, "csrc", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_DEPENDS = [MARSHAL_SOURCE, os.path.join(ROOT, "include", "sdv.h")]  # the header's structs are compiled into it

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # packed fp32 instructions stay off: plain fp32 code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(cmd: list, what: str) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {what} ({res.returncode}):\n{res.stderr}")
    return res.stderr


def build_library(out: str = LIBRARY, verbose: bool = False) -> str:
    hipcc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory() as where:
        objects = [os.path.join(where, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=8) as pool:
            said = list(pool.map(lambda job: _compile([hipcc, *HIPCC_FLAGS, f"-I{os.path.join(ROOT, 'include')}", "-c",
                                                       job[0], "-o", job[1]], job[0]), zip(SOURCES, objects)))
        # a name without a directory, by which what is linked with the library finds it
        said.append(_compile([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", f"-Wl,-soname,{os.path.basename(LIBRARY)}",
                              *objects, "-o", tmp], out))
    if verbose and any(said):
        print("".join(said))
    os.replace(tmp, out)
    return out


def build_marshal(out: str = MARSHAL) -> str:
    """_marshal.so, beside libsdv.so, which it is linked with and which it loads from its own directory."""
    import sysconfig

    import torch
    where = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    includes = [os.path.join(where, "include"), os.path.join(where, "include", "torch", "csrc", "api", "include"),
                os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    tmp = out + ".tmp"
    _compile(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
              *[x for i in includes for x in ("-isystem", i)], MARSHAL_SOURCE, "-o", tmp,
              f"-L{os.path.join(where, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_hip",
              f"-L{PKG}", f"-l:{os.path.basename(LIBRARY)}", "-Wl,-rpath,$ORIGIN"], MARSHAL_SOURCE)
    os.replace(tmp, out)
    return out


def is_stale(path: str | None = None) -> bool:
    """Whether a library at `path`, or with none given the library or the module, is missing or older than its sources."""
    if path is None:
        return is_stale(LIBRARY) or _older(MARSHAL, MARSHAL_DEPENDS)
    return _older(path, DEPENDS)


def _older(path: str, sources: list) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in sources)


if __name__ == "__main__":
    print(build_library(verbose=True), build_marshal())
