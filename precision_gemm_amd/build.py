"""Build the HIP library ``liblora_lowp.so`` in-tree for gfx950 with hipcc, and the attention
block's Python binding ``_attn.so`` that links to it.

Run as ``python -m precision_gemm_amd.build``; ``__graft_entry__.build()`` calls
:func:`build`.  Every call compiles (no up-to-date check), so a changed source is
always picked up.
"""

from __future__ import annotations

import json
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblora_lowp.so")
SOURCES = ["lora_kernels.hip", "lora_gemm_pf.hip", "lora_backward.hip", "lora_api.cpp"]
# the attention block, apart from the layer's sources (whose hash names the layer's profiles)
CSRC_ATTN = os.path.join(HERE, "csrc_attn")
SOURCES_ATTN = ["rope_kernels.hip", "tree_attention.hip", "attn_api.cpp"]
ARCH = "gfx950"

# -packed-fp32-ops off: no v_pk_{add,mul,fma}_f32 in the device code.
# atomic optimizer off: it rewrites a single-lane atomic with return into a wave-level
# scan whose result is consumed at once, which forces a wait for every load in flight.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
    "-Wno-unused-result",
    # per-kernel register, scratch and LDS use, kept next to the library (see resources())
    "-Rpass-analysis=kernel-resource-usage",
]
RESOURCES = LIB + ".resources.json"
BINDING = os.path.join(HERE, "_attn.so")


def parse_resources(stderr: str) -> dict:
    """Per-kernel resource use from the compiler's kernel-resource-usage remarks."""
    out, cur = {}, None
    for line in stderr.splitlines():
        if "[-Rpass-analysis=kernel-resource-usage]" not in line:
            continue
        body = line.split("remark:", 1)[1].rsplit("[-Rpass", 1)[0].strip()
        key, _, val = body.partition(":")
        key, val = key.strip(), val.strip()
        if key == "Function Name":
            cur = out.setdefault(val, {})
        elif cur is not None:
            cur[key] = int(val) if val.lstrip("-").isdigit() else val
    return out


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *FLAGS, "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES],
           *[os.path.join(CSRC_ATTN, s) for s in SOURCES_ATTN]]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    lines = [l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l]
    errs = "\n".join(l for l in lines if "kernel-resource-usage" not in l and not l.lstrip().startswith(("|", "^"))
                     and not l.strip().isdigit())
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{errs}")
    if verbose and errs.strip():
        print(errs, file=sys.stderr)
    os.replace(tmp, LIB)
    with open(RESOURCES, "w") as f:
        json.dump(parse_resources(res.stderr), f, indent=1, sort_keys=True)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """The attention block's binding (host code against the installed torch), beside the library
    it calls."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-I{p}" for p in include_paths()], "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC_ATTN, "binding.cpp"), "-o", tmp, f"-L{HERE}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           *[f"-L{p}" for p in library_paths()], "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding's compilation failed ({res.returncode}):\n{res.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def resources() -> dict:
    """Resource use of every kernel of the last build (empty if none was recorded)."""
    try:
        with open(RESOURCES) as f:
            return json.load(f)
    except OSError:
        return {}


if __name__ == "__main__":
    print(build(verbose=True))
