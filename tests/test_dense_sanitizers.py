"""The dense operators' host layer -- argument validation, the choice of kernel and shares,
workspace sizes -- built host-only with AddressSanitizer and UndefinedBehaviorSanitizer,
linked with stand-ins for the launches and driven over sizes from 0 to the limits
(tests/native/dense_abi_check.cpp)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_dense_host_layer_under_asan_ubsan(tmp_path):
    exe = tmp_path / "dense_abi_check"
    cmd = [HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-std=c++17",
           "-ffp-contract=off",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined",
           "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(ROOT, "trellis_coded_weight_amd", "csrc"), "-o", str(exe),
           os.path.join(ROOT, "trellis_coded_weight_amd", "csrc", "qtcq_dense.hip"),
           os.path.join(HERE, "native", "dense_abi_check.cpp")]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=1:abort_on_error=1"
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
