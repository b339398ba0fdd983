"""The host code of the RMS norm and of the 8-bit layer under AddressSanitizer and UndefinedBehaviorSanitizer:
tests/abi_q8_check.cpp linked with their sources and eql_api.hip rebuilt with the sanitizers
on their host code only, and with the library's other objects.  Runs on the CPU."""
import os
import subprocess

import pytest

from group_circulant_linear_p4_amd import build as B
from test_abi_sanitized import SAN, SAN_FLAGS, _run


def test_q8_abi_host_code_under_asan_and_ubsan():
    checked = ("eql_api.hip", "eql_block_api.hip", "eql_q8_api.hip")
    others = [os.path.join(B.BUILD, os.path.splitext(s)[0] + ".o") for s in B.SOURCES if s not in checked]
    if any(not os.path.exists(o) for o in others):
        pytest.skip("library objects not built (run the full build first)")
    os.makedirs(SAN, exist_ok=True)
    flags = [f for f in B.CFLAGS if f != "-O3"] + ["-O1"] + SAN_FLAGS
    here = os.path.dirname(os.path.abspath(__file__))
    objs = []
    for name, src in ((os.path.splitext(s)[0], os.path.join(B.CSRC, s)) for s in checked):
        objs.append(os.path.join(SAN, name + "_q8.o"))
        _run([B.hipcc(), *flags, "-c", src, "-o", objs[-1]])
    objs.append(os.path.join(SAN, "abi_q8_check.o"))
    _run([B.hipcc(), *flags, "-x", "hip", "-c", os.path.join(here, "abi_q8_check.cpp"), "-o", objs[-1]])
    exe = os.path.join(SAN, "abi_q8_check")
    _run([B.hipcc(), "--offload-arch=" + B.ARCH, *SAN_FLAGS, *objs, *others, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and ", 0 failed" in res.stdout, out[-6000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-6000:]
