"""CPU checks of the binding of what stands around the experts: what it hands on is what its objects say."""

import ctypes

import pytest
import torch

from top_routing_grouped_gemm_gb300 import moe


@pytest.mark.parametrize("field, value", [("score", moe.MOE_SCORE_SOFTMAX), ("groups", 8), ("groups_kept", 4),
                                          ("group_best", 2), ("renormalise", False), ("scale", 2.5)])
def test_a_rule_that_is_changed_is_what_the_library_reads(field, value):
    rule = moe.RouteRule(moe.MOE_SCORE_SIGMOID)
    before = moe.moe_route_rule.from_address(rule.c())
    assert [getattr(before, n) for n, _ in before._fields_] == [1, 1, 1, 1, 1, 1.0]
    setattr(rule, field, value)
    assert getattr(rule, field) == value
    assert getattr(moe.moe_route_rule.from_address(rule.c()), field) == value


def test_a_rule_by_position():
    rule = moe.RouteRule(moe.MOE_SCORE_SIGMOID, 8, 4, 2, False, 2.5)
    assert [getattr(rule, n) for n, _ in moe.moe_route_rule._fields_] == [1, 8, 4, 2, 0, 2.5]
    assert ctypes.sizeof(rule) == ctypes.sizeof(moe.moe_route_rule)


@pytest.mark.parametrize("group", [0, -32])
def test_packing_refuses_groups_of_nothing(group):
    codes, scales = torch.zeros(1, 16, 32, dtype=torch.uint8), torch.zeros(1, 16, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="codes|scales"):
        moe.moe_w4_pack(1, 16, 64, group, codes, scales, None, codes, codes)
    with pytest.raises(ValueError, match="codes|scales"):
        moe.W4Weights(torch.zeros(1, 16, 0, dtype=torch.uint8), scales)


def test_weights_whose_arrays_are_replaced_are_what_the_library_reads():
    """A copy made elsewhere, say, of arrays that are then given up."""
    w = object.__new__(moe.W4Weights)
    w.E, w.rows, w.cols, w.group, w.has_zeros = 2, 16, 64, 32, True
    w.codes, w.scales = (torch.zeros(n, dtype=torch.uint8) for n in (1024, 256))
    for _ in range(2):
        read = moe.moe_w4.from_buffer_copy(w.c("w", (2, 16, 64), -1))
        assert [getattr(read, n) for n, _ in read._fields_] == [w.codes.data_ptr(), w.scales.data_ptr(), 32, 1]
        w.codes, w.scales = w.codes.clone(), w.scales.clone()
    assert ctypes.sizeof(moe.moe_w4) == moe._W4.size


def test_selftest_of_the_4_bit_experts_waits_refuses():
    lib = moe.lib()
    for args in ((2001, 0, 0, 0, 0), (-1, 0, 0, 0, 0), (5, 0, -1, 0, 0), (5, 0, 0, -1, 0), (5, 1, 0, 0, -1)):
        assert lib.moe_selftest_w4_waits(*args) == 1
    p = moe.Problem(T=4, d=64, E=4, k=2, F=64)
    try:
        moe.moe_selftest_w4_waits(5)
        for group, zeros in ((64, 0), (32, 1)):  # (addresses that nothing reads)
            w4 = moe.moe_w4(0x10000, 0x10000, group, zeros)
            m = ctypes.addressof(w4)
            assert lib.moe_w4_expert_ffn(p.c(), *[0x10000] * 3, m, m, m, 0x10000, 0x10000, 1 << 40, None,
                                         None) == 2
    finally:
        moe.moe_selftest_w4_waits(0)
