"""Builds libqgemm.so (the HIP kernels and the C ABI of include/qgemm.h) for gfx950 with hipcc.

Every source is compiled in parallel to an object, then linked into
block_quantized_weight_affine_amd/libqgemm.so (in-tree, so it travels with the repository).
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libqgemm.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = ["qg_gemm.hip", "qg_gemv.hip", "qg_moe.hip", "qg_misc.hip", "qg_kv8.hip", "qg_kv8_rope.hip", "qg_attn8.hip",
           "qg_attn8_tile.hip", "qg_attn8_tree.hip", "qg_attn8_tree_tile.hip", "qg_draft.hip", "qg_w8a8.hip", "qg_capi.cpp",
           "qg_capi8.cpp"]
ARCH = os.environ.get("QG_OFFLOAD_ARCH", "gfx950")

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed-FP32 instructions stay disabled in every HIP object
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-rdc", "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]

# the attention kernels' sums stay in vector registers, where the softmax works on them, as far as those go: 16-bit
# tiles with heads of 192 and 256 and f32 tiles from 96 on keep 10 to 220 of theirs in accumulation registers
_SUMS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
EXTRA = {src: _SUMS for src in ("qg_attn8.hip", "qg_attn8_tile.hip", "qg_attn8_tree.hip", "qg_attn8_tree_tile.hip")}


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    cmd = ["hipcc", *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        # keep warnings visible, minus the host pass's note about the GPU-only target feature
        lines = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
        if lines:
            sys.stderr.write("\n".join(lines) + "\n")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    cmd = ["hipcc", "-shared", f"--offload-arch={ARCH}", "-fPIC", "-o", LIB + ".tmp", *objs]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
