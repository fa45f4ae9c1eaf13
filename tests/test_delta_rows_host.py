"""CPU test: where the gated delta rule looks for a sequence's rows and chunks
(csrc/delta.h, which the kernels use as it is), built with g++ under the
undefined-behaviour sanitizer and driven with rising, falling, negative and
extreme offsets (tests/host/rows.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_state_space_dplr_amd", "csrc")
HOST = os.path.join(ROOT, "tests", "host")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_rows_and_slots(tmp_path):
    exe = str(tmp_path / "rows")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-I", "/opt/rocm/include", os.path.join(CSRC, "token_api.cpp"),
           os.path.join(HOST, "token_stubs.cpp"), os.path.join(HOST, "rows.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "ok" in run.stdout


@pytest.mark.parametrize("sequences,tokens,most", [
    (1, 1, 1 << 10), (16, 16, 1 << 10), (128, 128, 16 << 20), (4096, 4096, 1 << 29),
    (16384, 16384, 3 << 29), (128, 1024, 128 << 20)])
def test_workspace_of_short_sequences(sequences, tokens, most):
    """Single tokens (bf16, 8 key and 16 value heads of 128 x 128) leave a workspace for what may
    still be long, not a chunk of 1.2 MB each."""
    import structured_state_space_dplr_amd as s4
    plan = s4.DeltaPlan(sequences, tokens, 8, 16, 128, 128, device="cpu")
    assert 0 < plan.workspace_bytes <= most
    assert plan.workspace().numel() >= plan.workspace_bytes if most < 1 << 20 else True
    trained = s4.DeltaPlan(sequences, tokens, 8, 16, 128, 128, training=True, device="cpu")
    assert trained.workspace_bytes > sequences * (1 << 20) and trained.saved_bytes > 0
