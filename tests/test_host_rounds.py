"""The norm-and-rotation kernels' walk over the tokens on the CPU (no GPU):
tests/plan/rounds_check.cpp against the header that the kernels use."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "plan", "rounds_check.cpp")
CSRC = os.path.join(ROOT, "tensor_adamw_optimizer_amd", "csrc")


def _run(tmp_path, include):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "rounds_check")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra",
                           "-fsanitize=undefined", "-fno-sanitize-recover=all",
                           "-I", str(include), "-o", exe, SRC])
    return subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                          timeout=120)


def test_every_token_once_up_to_the_largest_count(tmp_path):
    res = _run(tmp_path, CSRC)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout[-2000:]


def test_the_check_finds_a_position_that_overflows(tmp_path):
    text = open(os.path.join(CSRC, "ops_rounds.hpp")).read()
    old = "return tokens - t0 > step ? t0 + step : tokens;"
    assert text.count(old) == 1
    (tmp_path / "ops_rounds.hpp").write_text(text.replace(old, "return t0 + step + 0 * tokens;"))
    assert _run(tmp_path, tmp_path).returncode != 0


def test_the_kernels_walk_by_it():
    text = open(os.path.join(CSRC, "ops_qk_norm_rope.hip")).read()
    assert text.count("t0 = next_round(t0, ") == 2 and "t0 +=" not in text
