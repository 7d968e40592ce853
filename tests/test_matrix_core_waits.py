"""The listings of the matrix-core kernels of the decode window, as the
compiler writes them with the library's flags: no instruction reads a
v_mfma's result before enough wait states have passed, on any path.

The hardware does not hold such a read back; the compiler counts the wait
states, 8 for the 16x16x32 instructions on gfx950 (what it leaves in straight
lines of these listings at the least), and an early read gives wrong sums with
no other sign.
"""
import concurrent.futures as cf
import importlib.util
import os
import re
import subprocess

import pytest

from conftest import ROOT

WAIT = 8
PKG = os.path.join(ROOT, "row_gemv_decode_amd")


def registers(operands):
    out = set()
    for m in re.finditer(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", operands):
        out |= {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))
    return out


def early_reads(lines):
    """(v_mfma, early reader) pairs of one kernel's listing."""
    code, labels = [], {}
    for line in lines:
        text = line.split(";")[0].strip()
        m = re.match(r"(\.L\w+):", text)
        if m:
            labels[m[1]] = len(code)
        elif text and line[:1].isspace() and not text.startswith("."):
            op, _, args = text.partition(" ")
            code.append((op, args.strip()))

    def after(i):
        op, args = code[i]
        if op == "s_endpgm":
            return []
        if op == "s_branch":
            return [labels[args]]
        return [i + 1] + ([labels[args]] if op.startswith("s_cbranch") else [])

    found = []
    for i, (op, args) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        result = registers(args.split(", ")[0])
        todo, seen = [(j, 0) for j in after(i)], {}
        while todo:
            j, waited = todo.pop()
            if j >= len(code) or waited >= WAIT or seen.get(j, WAIT) <= waited:
                continue
            seen[j] = waited
            other, rest = code[j]
            if other.startswith("v_mfma"):
                d, a, b, c = (registers(x) for x in rest.split(", ")[:4])
                if (a | b) & result or (c & result and c != result):
                    found.append((code[i], code[j]))
                    continue
                if d == result:
                    continue  # the sum goes on in place
            elif other.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")) and registers(rest) & result:
                found.append((code[i], code[j]))
                continue
            waited += int(rest, 0) + 1 if other == "s_nop" else 1
            todo += [(k, waited) for k in after(j)]
    return found


STRAIGHT = """
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]
\ts_nop 7
\tv_add_f32_e32 v4, v4, v0
\ts_endpgm
"""
BEHIND_A_BRANCH = """
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]
\ts_cbranch_scc1 .LBB0_2
\ts_nop 7
.LBB0_2:
\tv_add_f32_e32 v4, v4, v0
\ts_endpgm
"""
OVER_A_LOOPS_END = """
.LBB0_1:
\tds_write_b128 v20, v[0:3]
\ts_nop 7
\tv_mfma_f32_16x16x32_f16 v[4:7], v[8:11], v[12:15], v[4:7]
\tv_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], v[0:3]
\ts_cbranch_scc0 .LBB0_1
\ts_endpgm
"""


@pytest.mark.parametrize("listing,reads", [(STRAIGHT, 0), (STRAIGHT.replace("s_nop 7", "s_nop 6"), 1), (BEHIND_A_BRANCH, 1),
                                           (OVER_A_LOOPS_END, 1)])
def test_early_reads_are_found(listing, reads):
    assert len(early_reads(listing.splitlines())) == reads


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    spec = importlib.util.spec_from_file_location("_skinny_build", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("listings")

    def listing(source):
        path = os.path.join(out, source + ".s")
        subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", os.path.join(PKG, "csrc", source), "-o", path],
                       check=True, capture_output=True)
        with open(path) as f:
            return f.read()

    with cf.ThreadPoolExecutor() as ex:
        return dict(zip(("moe.hip", "w4.hip"), ex.map(listing, ("moe.hip", "w4.hip"))))


@pytest.mark.parametrize("source,kernels", [("moe.hip", 50), ("w4.hip", 36)])
def test_no_kernel_reads_the_matrix_core_early(listings, source, kernels):
    parts = re.split(r"\n(_Z\w+):", listings[source])
    with_mfma = 0
    for name, body in zip(parts[1::2], parts[2::2]):
        body = body.split(".Lfunc_end")[0]
        with_mfma += "v_mfma" in body
        assert early_reads(body.splitlines()) == [], name
    assert with_mfma == kernels
