"""The compiled latent kernels that take the weights in two products
(latent_wide): what tests/test_attn_build.py demands of attn_latent."""
import os
import re
import subprocess

import pytest

import test_attn_build as base


@pytest.fixture(scope="module")
def wide(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "latent.s")
    subprocess.check_call([base._hipcc(), "-x", "hip", os.path.join(base.CSRC, "attn_latent.hip"), "-o", out,
                           "--cuda-device-only", "-S", "-w"] +
                          [f for f in base.hip_build.HIP_FLAGS if f not in ("-Wall", "-Wextra")])
    kernels, now, by_hand = {}, None, False
    for line in open(out):
        m = re.match(r"^(_Z\w*latent_wide\w*):", line)
        if m:
            now = kernels.setdefault(m.group(1), [])
        elif line.startswith(".Lfunc_end"):
            now = None
        if "#ASMSTART" in line or "#ASMEND" in line:
            by_hand = "#ASMSTART" in line
        text = line.split(";")[0].strip()
        if now is not None and text and not text.startswith(".") and not text.endswith(":"):
            now.append((text.split()[0], text[len(text.split()[0]):].strip(), by_hand))
    assert len(kernels) == 8, sorted(kernels)
    return kernels


@pytest.mark.parametrize("check", ["test_latent_outputs_have_their_registers_alone", "test_latent_products_read_settled_operands",
                                   "test_latent_scores_are_read_when_they_are_there", "test_no_packed_fp32"])
def test_latent_wide(wide, check):
    getattr(base, check)(wide)
