"""The host half of the low-bit entry points (``lowbit_api.cpp``) under
AddressSanitizer, UndefinedBehaviorSanitizer and ThreadSanitizer, on the CPU:
rebuilt with the sanitizers on the host side only and driven by
``lowbit_fuzz.cpp`` with seeded random calls, on one thread and on two."""

import os
import subprocess

import pytest

from test_host_sanitizers import COMMON, CSRC, HERE, INC, SAN, _hipcc, _run


@pytest.mark.timeout(900)
@pytest.mark.parametrize("kind", sorted(SAN))
def test_low_bit_host_code_is_clean_under_sanitizers(tmp_path, kind):
    if not os.path.exists(_hipcc()):
        pytest.skip("no hipcc")
    assert COMMON
    from zero_sharded_state_amd import build as B
    flags = [f for f in B.HIP_FLAGS if f not in ("-O3", "-fvisibility=hidden")] + ["-O1"]
    objs = []
    for src in ("api.cpp", "lowbit_api.cpp"):
        o = str(tmp_path / (src + ".o"))
        _run([_hipcc(), "-x", "hip", *flags, *SAN[kind], "-I", INC, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", o])
        objs.append(o)
    for name in ("kernels", "lowbit"):
        o = os.path.join(B.BUILD_DIR, name + ".o")
        if not os.path.exists(o):
            o = str(tmp_path / (name + ".o"))
            _run([_hipcc(), *B.HIP_FLAGS, "-I", INC, "-I", CSRC, "-c", os.path.join(CSRC, name + ".hip"), "-o", o])
        objs.append(o)
    drv = str(tmp_path / "fuzz.o")
    _run([_hipcc(), "-x", "c++", "-std=c++17", *SAN[kind], "-D__HIP_PLATFORM_AMD__", "-I", INC, "-I", "/opt/rocm/include", "-c",
          os.path.join(HERE, "lowbit_fuzz.cpp"), "-o", drv])
    exe = str(tmp_path / "fuzz")
    _run([_hipcc(), "--offload-arch=gfx950", *SAN[kind], *objs, drv, "-pthread", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1",
               TSAN_OPTIONS="halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    report = r.stdout + r.stderr
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), report[-4000:]
    for marker in ("ERROR: AddressSanitizer", "runtime error", "WARNING: ThreadSanitizer"):
        assert marker not in report, report[-4000:]
