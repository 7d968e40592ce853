"""The listings of the kernels of a batch of requests whose LDS is sized at the launch:
that part starts where the static one ends, and it is read 16 bytes at a time."""
import importlib.util
import os
import re
import subprocess

import pytest

from conftest import ROOT

PKG = os.path.join(ROOT, "row_gemv_decode_amd")


@pytest.mark.parametrize("source,kernels", [("adjust.hip", 48), ("adapters.hip", 61)])
def test_shared_memory_of_the_launch_starts_at_16_bytes(tmp_path, source, kernels):
    spec = importlib.util.spec_from_file_location("_skinny_build", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    path = os.path.join(tmp_path, source + ".s")
    subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", os.path.join(PKG, "csrc", source), "-o", path],
                   check=True, capture_output=True)
    with open(path) as f:
        sizes = [int(n) for n in re.findall(r"\.group_segment_fixed_size: (\d+)", f.read())]
    assert len(sizes) >= kernels and all(n % 16 == 0 for n in sizes)
