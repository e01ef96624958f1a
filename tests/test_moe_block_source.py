"""Rules of what stands around the experts that no run can show broken, checked in the source."""

import os
import re

import pytest

from test_sequence_mixing_source import body, source
from top_routing_grouped_gemm_gb300 import build as B

EARLY = [f for f in sorted(os.listdir(B.CSRC)) if '#include "overlap.cuh"' in source(f)]


@pytest.mark.parametrize("name", EARLY)
def test_kernels_set_up_early_wait_whatever_their_arguments(name):
    """What the kernel before the one before has written is there for a kernel after its own wait only."""
    code = source(name)
    waits = [line for line in code.splitlines() if "after_previous()" in line]
    assert waits and all(line.strip() == "after_previous();" for line in waits), waits


def test_products_of_4_bit_weights_wait_before_they_read():
    code = source("w4_experts.cu")
    for name in ("void run(", "void run_strips("):
        text = body(code, name)
        wait = text.index("after_previous();")
        assert text.count("after_previous();") == 1
        for read in ("p.g.chunks()", "p.g.good(", "Ahead ahead(", "AheadInStrips ahead("):
            assert read not in text or wait < text.index(read), (name, read)
