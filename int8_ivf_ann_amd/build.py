"""Build step for the gfx950 search library: compiles csrc/ with hipcc into libsvt.so (in-tree)."""
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsvt.so")
ARCH = "gfx950"
# packed-fp32 instructions are kept out of every kernel (the host pass warns that it does not know
# the feature; that warning is harmless)
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
# (source, holds device code); svt_api.cpp is host-only
SOURCES = (("svt_kernels.hip", True), ("svt_tile.hip", True), ("svt_noalloc.hip", True), ("svt_rerank.hip", True),
           ("svt_largek.hip", True), ("svt_api.cpp", False), ("experts/svt_route.hip", True),
           ("experts/svt_exchange.hip", True), ("experts/svt_quant.hip", True),
           ("experts/svt_linear_f32.hip", True), ("experts/svt_linear_f16.hip", True),
           ("experts/svt_linear_bf16.hip", True), ("scorer/svt_embedding.hip", True), ("scorer/svt_logprobs.hip", True),
           ("scorer/svt_gated.hip", True), ("scorer/svt_gated_f32.hip", True), ("scorer/svt_gated_f16.hip", True),
           ("scorer/svt_gated_bf16.hip", True))
COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result", "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory(prefix="svt_build_") as td:
        def compile_one(source):
            src, dev = source
            obj = os.path.join(td, src.replace("/", "_") + ".o")
            cmd = [hipcc] + COMMON + ["-c", os.path.join(CSRC, src), "-o", obj]
            if dev:
                cmd += ["--offload-arch=" + ARCH] + DEVICE_FLAGS
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            return obj

        with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as pool:
            objs = list(pool.map(compile_one, SOURCES))
        cmd = [hipcc, "-shared", "-fPIC", "--offload-arch=" + ARCH] + objs + ["-o", LIB + ".tmp", "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
