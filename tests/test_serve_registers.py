"""Registers of the serving kernels, from the metadata of the built library (CPU only)."""
import re

import pytest

from sparse_matrix_vector_amd import _lib as L
from test_attn_registers import device_images, kernels

pytest.importorskip("msgpack")


def test_two_blocks_a_cu_and_no_sums_in_memory():
    """Up to 128 columns: 256 ordinary registers, no accumulation registers, and no more than a few lane constants in
    scratch memory, whose loads would wait for the cache's."""
    with open(L.LIB_PATH, "rb") as f:
        data = f.read()
    seen = 0
    for image in device_images(data):
        for k in kernels(image):
            m = re.search(r"(13prompt_kernelILi\dELi|13shared_kernelILi\dELi\d+ELi|11tree_kernelILi\dELi\d+ELi)(\d+)E", k[".name"])
            if not m or int(m.group(2)) > 128:
                continue
            seen += 1
            assert k[".agpr_count"] == 0 and k[".vgpr_count"] <= 256, k[".name"]
            assert k[".vgpr_spill_count"] <= 8, (k[".name"], k[".vgpr_spill_count"])
    # prompts: two types, two widths, with and without lse; trees: two types, three formats, two widths, two of each form
    assert seen == 8 + 24 + 24
