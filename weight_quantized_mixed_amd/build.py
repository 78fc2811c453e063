"""Build libqgemm.so (hipcc, gfx950) and the module _binding.so (the host compiler) in-tree.

    python -m weight_quantized_mixed_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqgemm.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["api.hip", "pack.hip", "gemv.hip", "gemv16.hip", "mfma.hip", "mfma_dl.hip", "mfma_dl_gated.hip", "mfma_dl_rows.hip", "mfma_big.hip", "reduce.hip", "quant.hip", "gemv_mfma.hip", "gemv_mfma4.hip", "gated.hip",
           "kv_append.hip", "attention.hip", "attention_window.hip", "norm_rotate.hip", "kv_extend.hip"]

CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# packed fp32 vector ops are disabled for every device pass
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
COMMON = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # the host pass does not know the device feature flag: drop that notice only
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    return out


def build_binding() -> str:
    """The Python module that takes tensors to the C ABI (csrc/binding.cpp), against the installed PyTorch."""
    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [os.path.join(ROOT, "include"), *include_paths(), sysconfig.get_paths()["include"]]
    out = _run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-Wno-unused-variable",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include[:1]),
                *(x for d in include[1:] for x in ("-isystem", d)), os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp",
                f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-ltorch_cpu", "-ltorch_python"])
    os.replace(BINDING + ".tmp", BINDING)
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs = [os.path.join(BUILD, s.replace(".hip", ".o")) for s in SOURCES]

    def compile_one(i):
        src = os.path.join(CSRC, SOURCES[i])
        return _run([HIPCC, *COMMON, *DEVICE_FLAGS, "-c", src, "-o", objs[i]])

    # The library needs neither the host compiler nor PyTorch: it is linked whether or not the module can be built.
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding)
        outs = list(ex.map(compile_one, range(len(SOURCES))))
    tmp = LIB + ".tmp"
    outs.append(_run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]))
    os.replace(tmp, LIB)
    try:
        outs.append(binding.result())
    except (ImportError, OSError, RuntimeError) as e:  # no PyTorch; no compiler; no headers
        if os.path.exists(BINDING):  # (an older one would pass its arguments to a library that may take others)
            os.remove(BINDING)
        print(f"{os.path.basename(BINDING)} was not built, the calls that need it will say so: {e}", file=sys.stderr)
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
