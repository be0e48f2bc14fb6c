"""No kernel of the norm and its gradients spills vector registers: a row stays in them, so that each
tensor moves once."""

import os

import pytest

from mxfp4_quantized_expert_amd import binding
from tests.test_build_resources import code_objects, kernels


def test_no_vector_register_spills():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("the library is not built")
    with open(binding.LIB_PATH, "rb") as f:
        data = f.read()
    found = {k[".name"]: (k[".vgpr_spill_count"], k[".private_segment_fixed_size"])
             for elf in code_objects(data) for k in kernels(elf) if "rms_norm" in k[".name"]}
    assert len(found) >= 50  # the kernels were found at all
    assert not {n: c for n, c in found.items() if c != (0, 0)}
