"""Build the HIP library ``liblora_lowp.so`` in-tree for gfx950 with hipcc, and the Python bindings
that link to it: ``_attn.so`` (the attention block) and ``_step.so`` (norms and the AdamW step).

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
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblora_lowp.so")
SOURCES = ["lora_kernels.hip", "lora_gemm_pf.hip", "lora_backward.hip", "lora_api.cpp"]
# the attention block, apart from the layer's sources (whose hash names the layer's profiles)
CSRC_ATTN = os.path.join(HERE, "csrc_attn")
SOURCES_ATTN = ["rope_kernels.hip", "tree_attention.hip", "attn_api.cpp"]
# norms and the optimizer's step
CSRC_STEP = os.path.join(HERE, "csrc_step")
SOURCES_STEP = ["norm_kernels.hip", "adamw_kernels.hip", "step_api.cpp"]
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
BINDINGS = {os.path.join(HERE, "_attn.so"): os.path.join(CSRC_ATTN, "binding.cpp"),
            os.path.join(HERE, "_step.so"): os.path.join(CSRC_STEP, "binding.cpp")}


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


def _run(cmd: list, verbose: bool) -> str:
    """Run a compiler; its remarks (stderr), with anything else printed or raised."""
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
    return res.stderr


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    sources = [os.path.join(d, s) for d, names in ((CSRC, SOURCES), (CSRC_ATTN, SOURCES_ATTN), (CSRC_STEP, SOURCES_STEP))
               for s in names]
    compile_flags = [f for f in FLAGS if f != "-shared"]
    # a compiler a source, side by side: lora_kernels.hip takes as long as all others do one after another
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objs = [os.path.join(objects, f"{i}.o") for i in range(len(sources))]
        remarks = list(pool.map(lambda so: _run([hipcc(), *compile_flags, "-c", so[0], "-o", so[1]], verbose), zip(sources, objs)))
        _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    with open(RESOURCES, "w") as f:
        json.dump(parse_resources("\n".join(remarks)), f, indent=1, sort_keys=True)
    with ThreadPoolExecutor(len(BINDINGS)) as pool:
        list(pool.map(lambda b: build_binding(*b, verbose), BINDINGS.items()))
    return LIB


def build_binding(binding: str, source: str, verbose: bool = False) -> None:
    """A binding (host code against the installed torch), beside the library it calls."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = binding + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-I{p}" for p in include_paths()], "-I" + sysconfig.get_paths()["include"],
           source, "-o", tmp, f"-L{HERE}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           *[f"-L{p}" for p in library_paths()], "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_hip", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding's compilation failed ({res.returncode}):\n{res.stderr}")
    os.replace(tmp, binding)


def resources() -> dict:
    """Resource use of every kernel of the last build (empty if none was recorded)."""
    try:
        with open(RESOURCES) as f:
            return json.load(f)
    except OSError:
        return {}


if __name__ == "__main__":
    print(build(verbose=True))
