"""The host code of the bf16 / fp16 operators (ops.cpp: validation, sizes, workspace layout) under
AddressSanitizer and UndefinedBehaviorSanitizer: a g++ build with the launchers replaced by stand-ins
that write all of their scratch, driven by tests/sanitize/ops_driver.cpp (CPU only)."""
import os
import shutil

import pytest

from test_host_sanitizers import CSRC, FLAGS, ROCM, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")),
                    reason="needs g++ and the HIP runtime library")
def test_ops_host_code_under_asan_and_ubsan(tmp_path):
    hip = ["-L" + os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    drv = str(tmp_path / "ops_driver")
    src = [os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "ops.cpp")] + \
        [os.path.join(SAN, f) for f in ("launch_stubs.cpp", "ops_stubs.cpp", "ops_driver.cpp")]
    _run(["g++"] + FLAGS + src + ["-o", drv] + hip)
    r = _run([drv], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                             UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out and "LeakSanitizer" not in out, out
    assert "all statuses as expected" in out
