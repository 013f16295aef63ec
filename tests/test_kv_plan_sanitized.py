"""What kv_attention launches, on the host under AddressSanitizer and UndefinedBehaviorSanitizer: tests/host/kv_plan_checks.cpp
with the cache's C-ABI layer (csrc/kv_api.cpp), built with g++.  No GPU is involved."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers are missing")
    exe = tmp_path_factory.mktemp("kv_plan") / "kv_plan_checks"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
           os.path.join(ROOT, "block_quantized_decode_amd", "csrc", "kv_api.cpp"),
           os.path.join(ROOT, "tests", "host", "kv_plan_checks.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]

    def run(which):
        got = subprocess.run([str(exe), which], capture_output=True, text=True, timeout=120)
        assert got.returncode == 0, (got.stdout + got.stderr)[-4000:]
        assert f"{which} passed" in got.stdout
    return run


def test_window_never_takes_more_than_the_workspace_asked_for(checks):
    checks("window_workspace")


def test_windows_near_the_types_limit_reach_the_kernels_in_range(checks):
    checks("window_range")


def test_rows_of_a_head_are_refused_where_32_bits_do_not_count_them(checks):
    checks("row_count")


def test_batches_of_single_tokens_are_not_taken_for_prompts(checks):
    checks("unknown_rows")
