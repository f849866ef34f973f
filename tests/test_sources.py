"""Rules that the CUDA sources keep, checked on their text (no GPU needed)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(p for pattern in ("*.cu", "*.cuh", "*.h")
                 for p in glob.glob(os.path.join(ROOT, "nvfp4_block_scaled_route_gb300", "csrc", pattern)))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_is_multicast(path):
    """Processes on several GPUs load the one library, and callers choose the addresses
    that its TMA loads read: none of them is multicast to a cluster."""
    text = open(path).read()
    # the instruction may be spread over string literals
    text = re.sub(r'"\s*\n?\s*"', "", text)
    loads = re.findall(r"cp\.async\.bulk[^\s;\[]*", text)
    assert not [x for x in loads if "multicast" in x], path
    assert not re.search(r"\bmultimem\b|TENSOR_MAP.*MULTICAST", text), path


def test_the_sources_are_found():
    names = {os.path.basename(p) for p in SOURCES}
    assert {"attn_chunk.cu", "attn_rows.cu", "gemm.cu", "ptx.cuh"} <= names
