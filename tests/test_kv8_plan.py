"""Launch plans of the norm and 8-bit cache kernels (no GPU): every head and
token is covered, the gradient's partial rows fit its workspace, grids stay
within CUDA's limits."""
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_block_sparse_token_b200", "csrc")


@pytest.fixture(scope="module")
def rows():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["/usr/local/cuda/bin/nvcc", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
                        "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "native", "kv8_plan_check.cu"), "-o", exe], check=True,
                       capture_output=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    return [{k: int(v) for k, v in (f.split("=") for f in line.split())} for line in out.splitlines()]


def test_norm_grid(rows):
    seen = 0
    for r in (r for r in rows if r["kind"] == 0):
        seen += 1
        slots = (r["n"] + 31) // 32
        assert r["chunk"] >= 1 and r["qc"] * r["chunk"] >= r["hq"] and r["kc"] * r["chunk"] >= r["hkv"], r
        assert (r["qc"] - 1) * r["chunk"] < max(r["hq"], 1) and (r["kc"] - 1) * r["chunk"] < max(r["hkv"], 1), r
        assert 1 <= r["qc"] + r["kc"] <= 65535 and 1 <= r["x"] <= slots, r
        # token numbers are int32: the last round's start plus one more stride
        assert (r["x"] * 32) + r["n"] < 2 ** 31, r
        if r["back"]:
            assert (r["qc"] + r["kc"]) * r["x"] * 128 * 4 <= r["scratch"], r
        else:
            assert r["x"] == slots, r
    assert seen == 8 * 10 * 2


def test_pool_choice(rows):
    few = {(r["pairs"], r["blocks"]): r["few"] for r in rows if r["kind"] == 1}
    assert all(few[(p, 1)] for p in (1, 8, 37, 64, 128, 148, 512))
    assert few[(8, 16)] and not few[(64, 512)] and not few[(65535, 65535)] and not few[(8, 1 << 20)]
