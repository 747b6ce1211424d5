"""The validation of the linear products under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, on the CPU)."""
import os
import subprocess

import pytest

from test_layer_sanitizers import BASE, CSRC, HIPCC, ROOT, SAN


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.timeout(600)
def test_linear_validation_under_asan_and_ubsan(tmp_path):
    objs = []
    for src, flags in ((os.path.join(CSRC, "linear_abi.hip"), ["-O1", "-g"] + SAN),
                       (os.path.join(ROOT, "tests", "linear_validation_driver.cpp"), ["-O1", "-g"] + SAN),
                       (os.path.join(CSRC, "k_linear.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_linear_stream.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_linear_few.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_weight8.hip"), ["-O1"]),
                       (os.path.join(CSRC, "muon_abi.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_elementwise.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_ns_bf16.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_ns_f32.hip"), ["-O1"]),
                       (os.path.join(CSRC, "k_adamw.hip"), ["-O1"])):
        objs.append((src, flags, str(tmp_path / (os.path.basename(src) + ".o"))))
    jobs = [subprocess.Popen([HIPCC, *BASE, *flags, "-c", src, "-o", obj], stderr=subprocess.PIPE, text=True)
            for src, flags, obj in objs]
    for job in jobs:
        assert job.communicate()[1] is not None and job.returncode == 0
    exe = str(tmp_path / "driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN[:4], *[o for _, _, o in objs], "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ALL_VALIDATION_CASES_OK" in r.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
