"""The running calls' argument checks and size arithmetic under AddressSanitizer
and UndefinedBehaviorSanitizer, on the objects that the other calls' check
compiles (host code only, no GPU)."""
import os
import shutil
import subprocess

import pytest

from post_weight_quantization_layer_amd import build as LB
from tests import test_abi_sanitizers as S

DRIVER = os.path.join(S.ROOT, "tests", "sanitize", "run_checks.cpp")


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="needs hipcc")
def test_running_calls_under_asan_and_ubsan():
    objs = [os.path.join(S.OUT, s + ".o") for s in LB.SOURCES]
    heads = [os.path.join(LB.CSRC, "rows.h"), os.path.join(LB.INCLUDE, "gptq_run.h")]
    exe = S._build()
    newest = max(map(os.path.getmtime, heads))
    if not all(os.path.exists(o) and os.path.getmtime(o) >= newest for o in objs):
        os.remove(exe)               # made with other headers
        S._build()
    run = os.path.join(S.OUT, "run_checks")
    cmd = [LB.hipcc(), f"--offload-arch={LB.ARCH}", "-O1", "-g", "-std=c++17",
           "-fno-omit-frame-pointer", f"-I{LB.INCLUDE}", *S.SAN, "-x", "hip", DRIVER, "-x", "none",
           "-o", run, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([run], capture_output=True, text=True, env=env, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ok: 0 failure(s)" in out
    assert "runtime error" not in out and "AddressSanitizer" not in out
