"""The products' error words: a bit that is set while they are read and cleared is neither lost nor given twice."""
import os
import subprocess

import pytest

from mixture_experts_layer_35_b200 import build

pytestmark = pytest.mark.gpu


def test_no_error_is_lost_between_reading_and_clearing(tmp_path):
    exe = tmp_path / "error_words"
    subprocess.check_call([build._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-I",
                           build.INCLUDE, "-I", build.CSRC, "-o", str(exe),
                           os.path.join(os.path.dirname(__file__), "error_words.cu")], timeout=300)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout.split("\n")[:3]
    for line in lines:
        _, sets, _, taken = line.split()
        assert int(sets) > 1000 and sets == taken, lines
