"""Host code of the delta-rule layer under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the library built with
both sanitizers for the host side alone and linked into
tests/sanitize/layer_driver.cpp, which calls every entry point with
arguments that it must refuse (nothing is launched) and the workspace queries
over edge and extreme sizes.  A sanitizer report aborts the driver."""
import concurrent.futures as cf
import glob
import os

import pytest

from tests.test_sanitize import CSRC, ENV, HIPCC, HOST_SAN, ROCM_INCLUDE, ROOT, SAN, _run

UNITS = [os.path.basename(p)[:-4] for p in sorted(glob.glob(os.path.join(CSRC, "*.hip")))]


def test_layer_host_code_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    common = ["-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include")]
    flags = ["--offload-arch=gfx950", "-fPIC", "-I", CSRC, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    drv = str(tmp_path / "driver.o")
    jobs = [[HIPCC] + flags + common + HOST_SAN + ["-c", "-o", str(tmp_path / (u + ".o")), os.path.join(CSRC, u + ".hip")]
            for u in UNITS]
    jobs.append([HIPCC, "-x", "c++"] + common + ["-I", ROCM_INCLUDE, "-D__HIP_PLATFORM_AMD__"] + HOST_SAN +
                ["-c", "-o", drv, os.path.join(SAN, "layer_driver.cpp")])
    with cf.ThreadPoolExecutor(min(8, len(jobs))) as ex:
        for rc, out in ex.map(_run, jobs):
            assert rc == 0, out
    exe = str(tmp_path / "driver")
    rc, out = _run([HIPCC, "--offload-arch=gfx950"] + HOST_SAN + ["-o", exe, drv] +
                   [str(tmp_path / (u + ".o")) for u in UNITS])
    assert rc == 0, out
    rc, out = _run([exe], env=ENV, timeout=300)
    assert rc == 0, out[-4000:]
    assert "0 call(s) not rejected" in out
