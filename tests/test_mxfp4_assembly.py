"""Order of the matrix products that kernels_mxfp4.hip writes as inline assembly, in the
compiled code: the compiler sees no matrix instruction in them and puts no waits behind
them, so every read of an accumulator has to stand behind the kernel's own wait."""
import os
import re
import subprocess

import pytest

import pruning_quantization_amd.build as build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "mxfp4.s")
    r = subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, "kernels_mxfp4.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found, name = {}, None
    for line in open(out):
        head = re.match(r"(_Z\S*k_mxfp4_wide\S*):", line)
        if head:
            name = head.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and (text := line.split(";")[0].strip()):
            found[name].append(text)
    return found


def faults(code):
    """Reads and writes of accumulators outside the waits; (products, waits, faults)."""
    product = written = False  # since the last wait
    products = waits = 0
    wrong = []
    for prev, text in zip([""] + code, code):
        op = text.split()[0]
        if op == "s_nop" and text == prev == "s_nop 15":
            product = written = False
            waits += 1
        elif op.startswith("v_mfma"):
            products += 1
            product = True
            if written:
                wrong.append("product behind a write: " + text)
        elif re.search(r"\ba(\d|\[\d)", text):
            if product:
                wrong.append("accumulator ahead of the wait: " + text)
            written |= op.startswith("v_accvgpr")
    return products, waits, wrong


def test_accumulators_are_read_behind_the_wait(kernels):
    assert len(kernels) == 2
    for name, code in kernels.items():
        products, waits, wrong = faults(code)
        assert products >= 256 and waits >= 2, name
        assert not wrong, (name, len(wrong), wrong[:3])


def test_the_check_sees_what_it_is_for():
    mul, wait, read = "v_mfma_scale_f32 a[0:3], v[0:3], v[4:7], a[0:3]", ["s_nop 15", "s_nop 15"], "v_accvgpr_read_b32 v1, a1"
    assert faults([mul, *wait, read]) == (1, 1, [])
    assert faults([mul, read, *wait])[2] and faults([mul, "s_nop 15", read])[2]
    assert faults(["v_accvgpr_write_b32 a0, 0", mul])[2] and not faults(["v_accvgpr_write_b32 a0, 0", *wait, mul])[2]
