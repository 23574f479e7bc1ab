"""Build the gfx950 HIP library ``swiglu_mlp_amd/libck_convrot.so`` and, where
torch is installed, the Python extension ``swiglu_mlp_amd/_marshal.so`` in-tree.

Every translation unit is compiled by hipcc for gfx950 only, with
``-ffp-contract=off`` (the quantizer's FP32 steps must not be fused) and with
packed-FP32 instruction selection disabled.  Usage: ``python -m
swiglu_mlp_amd.build [--report]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libck_convrot.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
SOURCES = ["api.hip", "quant.hip", "gemm.hip", "gemm_big.hip", "gemm_blk.hip", "gemm_small.hip",
           "gemm_fused.hip", "qknorm.hip", "attn.hip", "attn_bf16.hip",
           "attn_fp16.hip", "probe.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str, obj_dir: str, report: bool) -> str:
    obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if report:
        cmd.append("-Rpass-analysis=kernel-resource-usage")
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(ln for ln in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in ln)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if report and out.strip():
        print(out)
    return obj


def _marshal() -> None:
    """The argument marshalling extension (host code, g++, torch's headers).
    Without torch there is none, and no caller for it: the library is for C."""
    try:
        import torch
    except ImportError:
        print(f"no torch: {os.path.basename(MARSHAL)} (the Python binding's extension) is not built")
        return
    home = os.path.dirname(torch.__file__)
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-o", tmp,
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on marshal.cpp:\n" + r.stdout + r.stderr)
    os.replace(tmp, MARSHAL)


def build(report: bool = False) -> str:
    obj_dir = os.path.join(ROOT, "_build", "ck")
    os.makedirs(obj_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_marshal)
        objs = list(ex.map(lambda s: _compile(s, obj_dir, report), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    r = subprocess.run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    marshal.result()   # its failure, with the library in place
    return LIB


if __name__ == "__main__":
    print(build(report="--report" in sys.argv))
