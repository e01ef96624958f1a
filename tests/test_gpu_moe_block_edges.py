"""What stands around the experts at its edges: experts out of range, infinite biases, calls from several
threads, outputs over inputs, orders and values next to a rounding.

Tolerances as in test_gpu_moe_block.py."""

import numpy as np
import pytest
import torch

from oracle import moe_block as MB
from parity_util import f64
from test_gpu_moe_block import BF, check_w4, w4_case
from top_routing_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ 4-bit experts

def guarded(n, dtype, fill=0x5A):
    """n bytes in the middle of a larger array of bytes `fill`, and whether those are as they were."""
    around = 1 << 20
    whole = torch.full((n + 2 * around,), fill, dtype=torch.uint8, device="cuda")
    return (whole[around:around + n].view(dtype),
            lambda: bool((whole[:around] == fill).all() and (whole[around + n:] == fill).all()))


def run_w4_guarded(case, w, x, idx, gate, status=None):
    """y, whose memory and the workspace's lie between bytes that no call may change."""
    T, d, E, k, F = case[:5]
    p = moe.Problem(T, d, E, k, F)
    packed = [moe.W4Weights(*(None if t is None else t.cuda() for t in m)) for m in w]
    ws, ws_kept = guarded(moe.moe_w4_expert_ffn_workspace_size(p), torch.uint8)
    y, y_kept = guarded(T * d * 2, BF)
    y = y.view(T, d)
    moe.moe_w4_expert_ffn(p, x.cuda(), idx.cuda(), gate.cuda(), *packed, y, ws, status)
    torch.cuda.synchronize()
    assert ws_kept() and y_kept()
    return y


BAD = {"first": [0], "middle": [1], "last": [-1], "first and last": [0, -1], "all": slice(None)}


# T, d, E, k, F, group, zeros, experts used; F far larger than d, and d than F
@pytest.mark.parametrize("where", BAD)
@pytest.mark.parametrize("case", [(1, 128, 5, 4, 1152, 64, True, None), (1, 64, 3, 3, 4096, 32, False, None),
                                  (1, 2048, 6, 5, 128, 128, True, None), (1, 512, 9, 8, 512, 128, False, None),
                                  (1, 64, 1, 1, 4096, 64, False, None), (1, 64, 40, 32, 256, 32, False, None)],
                         ids=str)
def test_w4_one_token_with_experts_out_of_range(case, where):
    """They contribute nothing and are reported; the others are as ever, time after time."""
    w, x, idx, gate = w4_case(case)
    bad = torch.zeros(case[3], dtype=torch.bool)
    bad[BAD[where] if case[3] > 1 else [0]] = True
    idx[0, bad] = torch.tensor([-1, case[2], 2 ** 31 - 1, -2 ** 31] * 8, dtype=torch.int32)[:int(bad.sum())]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = run_w4_guarded(case, w, x, idx, gate, status)
    assert int(status.item()) == 6
    check_w4(case, w, x, idx, gate, y)
    if where == "all":
        assert not y.any()
    for _ in range(10):
        assert torch.equal(run_w4_guarded(case, w, x, idx, gate), y)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("T", [1, 3])
def test_w4_experts_out_of_range_read_nobodys_weights(T, value):
    """What the experts that nobody names have for scales means nothing."""
    case = (T, 512, 6, 4, 256, 64, True, None)
    w, x, idx, gate = w4_case(case)
    idx[idx == 0] = 5
    idx[:, 1] = -1
    want = run_w4_guarded(case, w, x, idx, gate)
    for m in w:
        m[1][0] = value
    assert torch.equal(run_w4_guarded(case, w, x, idx, gate), want)
    assert not want.isnan().any()
