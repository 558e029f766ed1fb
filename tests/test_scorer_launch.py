"""Launch failures of the trained scorer's entry points, on the host: the stand-in for the runtime's launch calls (a
process of its own) counts the launches and fails the n-th; a call ends at the launch that fails."""
import os
import subprocess
import sys

import pytest

from test_experts_launch import CHILD, ROOT, STAND_IN

HEAD, TAIL = CHILD.split("CALLS = {")[0], CHILD.split("}\n", 1)[1]
CALLS = {
    "embedding": (1, "L.svt_embedding(64, 100, 24, 1, P[0], P[1], 1.0, P[2], None)"),
    "embedding_backward_one": (3, "L.svt_embedding_backward(64, 100, 24, 1, P[0], P[1], 1.0, 0, 1, P[2], P[3], 1 << 27, None)"),
    "embedding_backward_few": (2, "L.svt_embedding_backward(8, 100, 24, 1, P[0], P[1], 1.0, 0, 1, P[2], P[3], 1 << 27, None)"),
    "embedding_backward_two": (6, "L.svt_embedding_backward(100000, 100000, 24, 1, P[0], P[1], 1.0, 1, 0, P[2], P[3], 1 << 28, None)"),
    "embedding_backward_none": (1, "L.svt_embedding_backward(0, 100, 24, 1, None, None, 1.0, 0, 1, P[2], None, 0, None)"),
    "logprobs": (1, "L.svt_token_logprobs(600, 3000, 2, 0, P[0], P[1], 1.0, P[2], P[3], P[4], P[5], P[6], None, 0, None)"),
    "logprobs_split": (2, "L.svt_token_logprobs(2, 100000, 0, 0, P[0], P[1], 1.0, P[2], P[3], P[4], None, None, P[7], 1 << 20, None)"),
    "logprobs_backward": (1, "L.svt_token_logprobs_backward(4, 64, 2, P[0], P[1], 1.0, P[2], P[3], P[4], None, P[5], None)"),
    "gated_few": (1, "L.svt_gated_linear(8, 33, 16, 1, 1, P[0], P[1], P[2], None, 2, P[3], None, None, None, 0, None)"),
    "gated": (1, "L.svt_gated_linear(400, 32, 16, 1, 1, P[0], P[1], P[2], None, 2, P[3], P[4], P[5], None, 0, None)"),
    "gated_copies": (2, "L.svt_gated_linear(400, 33, 16, 1, 1, P[0], P[1], P[2], None, 2, P[3], P[4], P[5], P[6], 1 << 24, None)"),
    "gated_backward": (2, "L.svt_gated_linear_backward(400, 32, 16, 1, 1, P[0], P[1], P[2], P[3], P[4], P[5], None, 2, P[6], "
                          "P[7], P[7] + (1 << 27), 0xA0000000, 1 << 24, None)"),
    "gated_backward_parts": (4, "L.svt_gated_linear_backward(4000, 33, 2000, 1, 1, P[0], P[1], P[2], P[3], P[4], P[5], None, 2, "
                                "P[6], P[7], P[7] + (1 << 27), 0xA0000000, 1 << 28, None)"),
    "gated_backward_none": (1, "L.svt_gated_linear_backward(0, 32, 16, 1, 1, None, None, None, None, None, None, None, 2, None, "
                               "P[7], P[7] + (1 << 27), None, 0, None)"),
}


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    from int8_ivf_ann_amd import svt
    if not os.path.exists(svt.LIB_PATH):
        from int8_ivf_ann_amd import build
        build.build()
    d = tmp_path_factory.mktemp("launch")
    src, lib, child = d / "stand_in.c", d / "libstand_in.so", d / "child.py"
    src.write_text(STAND_IN)
    child.write_text(HEAD + "CALLS = {\n" + "".join(f"    {k!r}: ({n}, lambda: {c}),\n" for k, (n, c) in CALLS.items()) + "}\n" + TAIL)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    return str(lib), str(child)


@pytest.mark.parametrize("name", list(CALLS))
def test_a_failed_launch_ends_the_call(stand_in, name):
    lib, child = stand_in
    r = subprocess.run([sys.executable, child, lib, ROOT, name], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
