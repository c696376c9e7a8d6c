"""The layer operators' workspaces (growth, captures, clearing, release) on a fake CUDA runtime."""
from __future__ import annotations

import os
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]


def test_layer_scratch_on_a_fake_runtime(tmp_path):
    cxx = shutil.which("g++")
    include = Path(os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH") or "/usr/local/cuda") / "include"
    if cxx is None or not (include / "cuda_runtime.h").exists():
        pytest.skip("needs g++ and the CUDA headers")
    program = tmp_path / "layer_scratch_host"
    subprocess.run([cxx, "-std=c++17", "-O1", f"-I{include}", f"-I{ROOT / 'dense_fp32_gemm_08_gb300' / 'csrc'}",
                    str(ROOT / "tests" / "layer_scratch_host.cpp"), "-o", str(program), "-lpthread"],
                   check=True, timeout=300)
    run = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
