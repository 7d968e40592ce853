"""The listings of the adapters' matrix-core kernels: no instruction reads a v_mfma's
result before enough wait states have passed, on any path (see
test_matrix_core_waits, whose search this is)."""
import importlib.util
import os
import re
import subprocess

import pytest

from conftest import ROOT
from test_matrix_core_waits import early_reads

PKG = os.path.join(ROOT, "row_gemv_decode_amd")


def one_file(body):
    """Accumulation registers as vector registers from 512 on (the search knows v's only)."""
    body = re.sub(r"\ba\[(\d+):(\d+)\]", lambda m: f"v[{512 + int(m[1])}:{512 + int(m[2])}]", body)
    return re.sub(r"\ba(\d+)\b", lambda m: f"v{512 + int(m[1])}", body)


def test_early_reads_of_accumulation_registers_are_found():
    listing = """
\tv_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[12:15], a[0:3]
\ts_nop 6
\tv_accvgpr_read_b32 v4, a2
\ts_endpgm
"""
    assert len(early_reads(one_file(listing).splitlines())) == 1
    assert early_reads(one_file(listing.replace("s_nop 6", "s_nop 7")).splitlines()) == []


def test_no_adapter_kernel_reads_the_matrix_core_early(tmp_path):
    spec = importlib.util.spec_from_file_location("_skinny_build", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    path = os.path.join(tmp_path, "adapters.s")
    subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", os.path.join(PKG, "csrc", "adapters.hip"), "-o", path],
                   check=True, capture_output=True)
    with open(path) as f:
        parts = re.split(r"\n(_Z\w+):", f.read())
    with_mfma = 0
    for name, body in zip(parts[1::2], parts[2::2]):
        body = body.split(".Lfunc_end")[0]
        with_mfma += "v_mfma" in body
        assert early_reads(one_file(body).splitlines()) == [], name
        assert "scratch_" not in body, name  # (arrays that the compiler did not keep in registers)
    assert with_mfma >= 20
