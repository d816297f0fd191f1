"""The sizes planned on the host for adapters, weight gradients and the balance loss
(csrc/gemm_validate.hpp), under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil

import pytest

from test_sanitizers_cpu import CSRC, SAN, TESTS, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "plan_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-I", CSRC, os.path.join(TESTS, "plan_check.cpp"), "-o", exe], exe)
    assert " 0 failures" in out, out
