"""Host AddressSanitizer / UndefinedBehaviorSanitizer build of the fused products' checks and workspace plans.

As tests/test_host_sanitizers.py does for the other entry points: act_api.hip (with the shared checks of
aqlm_api.hip) on the host pass, tests/host_sanitize/act_validation_driver.hip in the place of every launcher.
"""
import os
import subprocess

from test_host_sanitizers import API, ROOT, _hipcc, _run

ACT_API = os.path.join(ROOT, "extreme_weight_quantization_amd", "csrc", "act_api.hip")
DRIVER = os.path.join(ROOT, "tests", "host_sanitize", "act_validation_driver.hip")


def _build(tmp_path, name, extra=()):
    exe = str(tmp_path / name)
    cmd = [_hipcc(), "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           *extra, API, ACT_API, DRIVER, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def test_fused_checks_are_clean_under_asan_and_ubsan(tmp_path):
    r = _run(_build(tmp_path, "act_check"))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "act validation ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr


def test_the_build_catches_a_planted_overread(tmp_path):
    r = _run(_build(tmp_path, "act_check_planted", ("-DAQLM_PLANT_OVERREAD",)))
    assert r.returncode != 0
    assert "heap-buffer-overflow" in r.stderr
