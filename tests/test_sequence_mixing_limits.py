"""CPU checks of the limits of the operators beside the gated delta rule: sizes and addresses that a
call refuses before anything reaches a GPU."""

import subprocess
import sys

import pytest

from conftest import ROOT
from top_routing_grouped_gemm_gb300 import build as B
from top_routing_grouped_gemm_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_workspace_size_of_widths_that_are_refused():
    """Widths below 8 are no reason to end the process (it is one of its own here), and a width that
    every call refuses has no workspace."""
    widths = [1, 4, 7, 12, 20, 250, 260]
    code = ("from top_routing_grouped_gemm_gb300 import moe\n"
            f"print([moe.moe_qk_norm_rope_backward_workspace_size(8, D, 4, 1) for D in {widths}])")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0, got.returncode
    assert got.stdout.strip() == str([0] * len(widths))
    assert all(moe.moe_qk_norm_rope_backward_workspace_size(8, D, 4, 1) > 0
               for D in range(8, 257, 8))


def test_selftest_of_the_recurrences_waits_refuses():
    for args in ((-1, 0, 0, 0), (2001, 0, 0, 0), (5, 0, 0, -1)):
        assert moe.lib().moe_selftest_recurrence_waits(*args) == 1
    assert moe.lib().moe_selftest_recurrence_waits(5, 0, 0, 0) == 0
    assert moe.lib().moe_selftest_recurrence_waits(0, 0, 0, 0) == 0
