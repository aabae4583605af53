"""Launches that are one wave of CTAs ask the device for its SMs: a share of the work per CTA is
fixed, so that a grid made for another number of SMs leaves some idle or runs a second wave."""
from __future__ import annotations

import os
import re

import pytest

from bit_asymmetric_kv_gb300 import build as kbuild


@pytest.mark.parametrize("source", ["kivi_packed_attention.cu", "kivi_packed_quant.cu", "kivi_pages.cu"])
def test_grids_follow_the_device(source):
    with open(os.path.join(kbuild.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\b(132|144|148|152|160)\b", code)  # SMs of a device as a number
    assert "device_sms(" in code
