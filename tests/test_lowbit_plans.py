"""Every launch of the low-bit entry points (``lowbit_api.cpp``) held against its
request on the CPU: ``lowbit_plans.cpp`` takes the place of the kernels'
launchers, so requests of many launches (more parameters, ranks or tensors than
one holds) run to their end, under AddressSanitizer and
UndefinedBehaviorSanitizer on the host side."""

import os
import subprocess

import pytest

from test_host_sanitizers import CSRC, HERE, INC, SAN, _hipcc, _run


@pytest.mark.timeout(900)
def test_every_launch_covers_its_request(tmp_path):
    if not os.path.exists(_hipcc()):
        pytest.skip("no hipcc")
    from zero_sharded_state_amd import build as B
    flags = [f for f in B.HIP_FLAGS if f not in ("-O3", "-fvisibility=hidden")] + ["-O1"]
    objs = []
    for src in (os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "lowbit_api.cpp"), os.path.join(HERE, "lowbit_plans.cpp")):
        o = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([_hipcc(), "-x", "hip", *flags, *SAN["asan+ubsan"], "-I", INC, "-I", CSRC, "-c", src, "-o", o])
        objs.append(o)
    kernels = os.path.join(B.BUILD_DIR, "kernels.o")
    if not os.path.exists(kernels):
        kernels = str(tmp_path / "kernels.o")
        _run([_hipcc(), *B.HIP_FLAGS, "-I", INC, "-I", CSRC, "-c", os.path.join(CSRC, "kernels.hip"), "-o", kernels])
    exe = str(tmp_path / "plans")
    _run([_hipcc(), "--offload-arch=gfx950", *SAN["asan+ubsan"], *objs, kernels, "-pthread", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    report = r.stdout + r.stderr
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), report[-4000:]
    for marker in ("ERROR: AddressSanitizer", "runtime error"):
        assert marker not in report, report[-4000:]
