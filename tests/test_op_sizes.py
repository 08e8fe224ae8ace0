"""The launch, tile and scratch sizes of the bf16 / fp16 operators (csrc/op_sizes.h) against counts made the
long way round by tests/sanitize/op_sizes_driver.cpp, under the sanitizers (CPU only)."""
import os
import shutil

import pytest

from test_host_sanitizers import CSRC, FLAGS, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_sizes_against_counts(tmp_path):
    drv = str(tmp_path / "op_sizes_driver")
    _run(["g++"] + FLAGS + [os.path.join(SAN, "op_sizes_driver.cpp"), "-o", drv])
    assert "all sizes as counted" in _run([drv]).stdout
