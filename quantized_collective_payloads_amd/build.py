"""Build libqcp.so (the gfx950 HIP library) in-tree.

    python -m quantized_collective_payloads_amd.build

Compiles each csrc/*.hip translation unit with hipcc for gfx950 in parallel and
links them into quantized_collective_payloads_amd/libqcp.so.  Flags that matter
for bit-exact results: -ffp-contract=off (no implicit FMA), correctly rounded
fp32 division, fp32 denormals kept, and packed-fp32 VALU instructions disabled.
The payloads' inputs are finite by contract, so the library is built without NaN
semantics (-fno-honor-nans, IEEE mode off): max/max3 then take |x| operands directly.
The files in HONOR_NANS promise something about NaN and keep its semantics.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqcp.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["qcp_api.hip", "qcp_codec.hip", "qcp_reduce.hip", "qcp_ops_api.hip", "qcp_adamw.hip",
           "qcp_mxfp4.hip", "qcp_mxfp4_matmul.hip", "qcp_int8.hip", "qcp_int8_matmul.hip", "qcp_int8_mixed.hip"]

NO_NANS = ["-fno-honor-nans", "-mno-amdgpu-ieee"]
HONOR_NANS = {"qcp_ops_api.hip", "qcp_adamw.hip", "qcp_mxfp4.hip", "qcp_mxfp4_matmul.hip", "qcp_int8.hip",
              "qcp_int8_matmul.hip", "qcp_int8_mixed.hip"}

CXXFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    *NO_NANS,
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    flags = [f for f in CXXFLAGS if not (f in NO_NANS and src in HONOR_NANS)]
    cmd = [HIPCC, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    print(LIB)
