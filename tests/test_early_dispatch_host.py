"""Kernels that are dispatched while their predecessor still runs live while it writes what they read.  Loads through the
non-coherent path (``__ldg``) want their data read-only for the kernel's whole life, so of these kernels' inputs only
the norm's weights, which no kernel of the library writes, may come that way."""

import os
import re

import pytest

import lm_head_linear_gb300.build as build

EARLY = ["norm_kernels.cuh", "fp8_kernels.cuh", "sample_kernels.cuh"]


@pytest.mark.parametrize("name", EARLY)
def test_only_weights_through_the_non_coherent_path(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    assert "wait_prerequisites" in text
    text = re.sub(r"void load_weight_pairs\(.*?\n}\n", "", text, flags=re.S)
    calls = [line.strip() for line in text.splitlines() if "__ldg(" in line or "ld.global.nc" in line or "__restrict__" in line]
    assert [c for c in calls if "(p.w)" not in c] == []
