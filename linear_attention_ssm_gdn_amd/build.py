"""Build libgdn.so (HIP kernels for gfx950 + the C ABI) in this directory.

Every translation unit is compiled by hipcc for gfx950 only, in parallel,
then linked into one shared library that exports the gdn_* symbols of
include/gdn.h, the gdnt_* symbols of include/gdn_train.h, the gdnl_* symbols of
include/gdn_linear.h and nothing else.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgdn.so")
OBJ = os.path.join(HERE, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["gdn_api.cpp", "gdn_seq.hip", "gdn_conv.hip", "gdn_verify.hip", "gdn_chunked.hip", "gdn_mixed.hip",
           "gdn_noalloc.hip", "gdnt_api.cpp", "gdnt_map.hip", "gdnt_scan.hip",
           "gdnt_scan_bwd.hip", "gdnt_conv.hip", "gdnl_api.cpp", "gdnl_segments.hip", "gdnl_attend_bf16.hip",
           "gdnl_attend_bf16_back.hip", "gdnl_attend_f32.hip", "gdnl_attend_f32_back.hip", "gdnl_tokens.hip", "gdnl_rotate.hip", "gdnl_cache.hip"]
FLAGS = [
    "--offload-arch=gfx950", "-mcode-object-version=5", "-O3", "-std=c++17", "-fPIC",
    "-fvisibility=hidden", "-ffp-contract=off", "-Wall", "-Wno-unused-function",
    # packed fp32 instructions stay off on the test machines
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
]


def _compile(src: str, verbose: bool) -> str:
    os.makedirs(OBJ, exist_ok=True)
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC] + FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msg}")
    if msg.strip() and verbose:
        print(msg, flush=True)
    return obj


def build(verbose: bool = False, jobs: int = 0) -> str:
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 4, 8)
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", LIB + ".tmp"] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
