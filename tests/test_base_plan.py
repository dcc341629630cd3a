"""The cut of a batch between the row-streaming and the tiled base products, on
the host: its arithmetic under sanitizers, and the query's refusals."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_cut_under_sanitizers(tmp_path):
    exe = tmp_path / "test_base_plan"
    src = os.path.join(ROOT, "tests", "cpp", "test_base_plan.cpp")
    inc = os.path.join(ROOT, "segmented_gathered_rank_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", inc, src, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "ok" in r.stdout


def test_tile_tokens_refuses_a_null_pool():
    import segmented_gathered_rank_amd as sgr
    assert sgr.lora_fused_tile_tokens(0, 0, 1, 4, 100, True) == -1
