"""CPU: the state space and beam search entry points in a host build of the
library under AddressSanitizer and UndefinedBehaviorSanitizer
(tests/sanitize/ssm_beam_driver.cpp; GPU code is not instrumented and nothing
reaches a device)."""
import concurrent.futures as fut
import glob
import os
import subprocess

import pytest

from tests.test_sanitizers import HERE, HIP_SAN, HIPCC, ROOT, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_new_entry_points_under_asan_and_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "gated_deltanet_decode_amd", "csrc")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-ffp-contract=off",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"), "-I", csrc]
    srcs = sorted(glob.glob(os.path.join(csrc, "*.hip"))) + [os.path.join(HERE, "ssm_beam_driver.cpp")]

    def compile_one(src):
        obj = tmp_path / (os.path.basename(src) + ".o")
        subprocess.run([HIPCC, *flags, *HIP_SAN, "-c", src, "-o", str(obj)], check=True, capture_output=True)
        return str(obj)

    with fut.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
        objs = list(pool.map(compile_one, srcs))
    exe = tmp_path / "ssm_beam_asan"
    subprocess.run([HIPCC, "--offload-arch=gfx950", *HIP_SAN, "-o", str(exe), *objs], check=True,
                   capture_output=True)
    r = _run(str(exe))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "every call refused as expected" in r.stdout
