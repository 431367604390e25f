"""The host side of the mixers' .hip files, built without device code and linked against a
recorder in place of the HIP runtime (tests/abi_host/launch_recorder.hpp): which kernels a call
launches, with what sizes.  No GPU is involved."""
import os
import shutil
import subprocess

import pytest

from nvfp4_w4a4_block_act_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HOST = os.path.join(ROOT, "tests", "abi_host")
ROCM_INCLUDE = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")


def recorded(tmp_path, program, *sources):
    """Builds and runs a program of tests/abi_host with the host code of .hip sources; its output."""
    gxx = shutil.which("g++")
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        hipcc = None
    if gxx is None or hipcc is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("g++, hipcc or the HIP runtime headers are not available")
    objects = []
    for src in sources:
        objects.append(str(tmp_path / (src + ".o")))
        subprocess.run([hipcc, "-std=c++17", "-O1", f"--offload-arch={build.ARCH}", "--offload-host-only", "-c",
                        os.path.join(build.CSRC, src), "-o", objects[-1]], check=True, capture_output=True, timeout=300)
    exe = str(tmp_path / "check")
    b = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
                        os.path.join(HOST, program), *objects, "-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files",
                        "-o", exe], capture_output=True, text=True, timeout=300)   # (unresolved: the device code)
    assert b.returncode == 0, b.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-4000:])
    assert r.stdout.strip().splitlines()[-1].startswith("ok "), r.stdout
    return r.stdout


def test_attention_launches(tmp_path):
    recorded(tmp_path, "check_attn_launch.cpp", "attn_decode.hip")


def test_attention_splits(tmp_path):
    recorded(tmp_path, "check_attn_splits.cpp")


def test_prefill_launches(tmp_path):
    recorded(tmp_path, "check_prefill_launch.cpp", "gdn_prefill.hip")
