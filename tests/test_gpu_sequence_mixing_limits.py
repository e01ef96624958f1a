"""GPU checks of the operators beside the gated delta rule at the limits of what their headers allow:
order in the stream off the fast paths, inputs of one shared row, waits that run out, batches of
mostly empty sequences, infinities."""

import numpy as np
import pytest
import torch

from oracle import sequence_mixing as SM
from top_routing_grouped_gemm_gb300 import moe
from parity_util import f64
from test_gpu_sequence_mixing import BF, CODE, F32, LAST, U, close, majorants

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype, D, wide", [(F32, 126, 129), (BF, 126, 130), (BF, 125, 127)])
def test_calls_off_16_byte_boundaries_keep_the_order_of_their_stream(dtype, D, wide, captured):
    """A chain in which every call reads what the one before it wrote has the bits of the same chain
    with a wait after every call, where rows are copied without TMA."""
    N, code = 200, CODE[dtype]
    gen = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(s, generator=gen).to(dtype).cuda()  # noqa: E731
    first = dict(g=-r(N, wide).abs(), x=r(N, wide), dg=r(N, wide), dx=r(N, wide), h=r(N, D),
                 h2=r(N, D), h_T=r(1, D).float(), c=r((N + 63) // 64, D).float())

    def chain(b, wait):
        part = {n: b[n][:, :D] for n in ("g", "x", "dg", "dx")}

        def forward(x, h):
            moe.moe_glr_forward(N, D, 1, None, moe.MOE_GLR_MIX, code, part["g"], part[x], b["h_T"],
                                b[h], b["h_T"], b["c"])

        def backward(x, dh):
            moe.moe_glr_backward(N, D, 1, None, moe.MOE_GLR_MIX, code, part["g"], part["x"], None,
                                 b["c"], b[dh], None, part["dg"], part["dx"], None)

        calls = [lambda: forward("x", "h"), lambda: backward("x", "h"), lambda: forward("dx", "h2"),
                 lambda: backward("x", "h2"), lambda: b["x"].copy_(b["dx"]).tanh_(),
                 lambda: forward("x", "h"), lambda: b["g"].copy_(b["dg"]).clamp_(-4, 0)]
        for _ in range(12):
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()

    want, got = ({n: t.clone() for n, t in first.items()} for _ in range(2))
    chain(want, True)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(got, False)
        for n, t in first.items():
            got[n].copy_(t)
        graph.replay()
    else:
        chain(got, False)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n].view(torch.int16), want[n].view(torch.int16)), n
