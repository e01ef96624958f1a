"""GPU checks of the operators beside the gated delta rule at the limits of what their headers allow:
order in the stream off the fast paths, inputs of one shared row, waits that run out, batches of
mostly empty sequences, infinities."""

import numpy as np
import pytest
import torch

from oracle import sequence_mixing as SM
from top_routing_grouped_gemm_gb300 import moe
from parity_util import f64
from test_gpu_sequence_mixing import BF, CODE, F32, close, majorants

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


@pytest.fixture
def impatient():
    """Ends the self-test of the waits whatever the test does."""
    yield
    moe.moe_selftest_recurrence_waits(0)


def training_pass(N, D, dtype, n_seq, seed):
    """(forward, backward, outputs) of one pass over sequences of equal length."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    g, x, dh = torch.nn.functional.logsigmoid(r(N, D) + 3).to(dtype), r(N, D).to(dtype), r(N, D).to(dtype)
    h0, dh_T = r(n_seq, D), r(n_seq, D)
    out = dict(h=torch.zeros_like(g), h_T=torch.zeros_like(h0), dg=torch.zeros_like(g),
               dx=torch.zeros_like(g), dh0=torch.zeros_like(h0),
               chunks=torch.zeros(((N + 63) // 64, D), device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    head = (N, D, n_seq, None, moe.MOE_GLR_MIX, CODE[dtype], g, x, h0)
    return (lambda: moe.moe_glr_forward(*head, out["h"], out["h_T"], out["chunks"], status),
            lambda: moe.moe_glr_backward(*head, out["chunks"], dh, dh_T, out["dg"], out["dx"],
                                         out["dh0"], status), out, status)


# rows, channels, type, sequences: clusters of 16 and of 8 blocks, single blocks, two sequences to a
# part; with TMA and without
@pytest.mark.parametrize("N, D, dtype, n_seq", [(9000, 64, BF, 1), (6000, 1024, F32, 1),
                                                (5000, 8 * 2048, BF, 1), (60, 40, F32, 1),
                                                (8000, 512, BF, 40), (7000, 62, BF, 1),
                                                (4000, 33, F32, 4)])
def test_scans_that_give_up_end_by_themselves_and_harm_nobody(N, D, dtype, n_seq, impatient):
    """One warp of a cluster leaves early, in every role and at several steps; all that wait for it
    run out of patience.  The launch ends, says so, and what runs beside it and after it has its
    bits."""
    forward, backward, out, status = training_pass(N, D, dtype, n_seq, 1)
    o_forward, o_backward, o_out, o_status = training_pass(3000, 520, F32, 3, 2)
    forward(), backward(), o_forward(), o_backward()
    want, o_want = ({n: t.clone() for n, t in o.items()} for o in (out, o_out))
    torch.cuda.synchronize()
    assert int(status) == 0 and int(o_status) == 0
    side = torch.cuda.Stream()
    tries = [(0, 0, 0), (1, 7, 1), (0, 8, 0), (2, 8, 1), (0, 9, 0), (3, 9, 2), (1, 8, 3), (0, 4, 2)]
    for call in (forward, backward):
        gave_up = 0
        for rank, warp, step in tries:
            status.zero_()
            for t in o_out.values():
                t.zero_()
            torch.cuda.synchronize()
            moe.moe_selftest_recurrence_waits(4, rank, warp, step)
            call()
            moe.moe_selftest_recurrence_waits(0)
            with torch.cuda.stream(side):
                o_forward(), o_backward()
            torch.cuda.synchronize()
            assert int(status) in (0, 5)  # MOE_ERR_TIMEOUT where there is such a block and step
            gave_up += int(status) == 5
            assert int(o_status) == 0
            assert all(torch.equal(o_out[n], o_want[n]) for n in o_want)
        assert gave_up >= 2
    status.zero_()
    for t in out.values():
        t.zero_()
    forward(), backward()
    torch.cuda.synchronize()
    assert int(status) == 0
    assert all(torch.equal(out[n], want[n]) for n in want)


@pytest.mark.parametrize("n_seq", [511, 512, 5000, 1 << 24])
def test_few_rows_among_millions_of_empty_sequences(n_seq):
    """However many sequences are empty, no wait runs out: rows have the bits of a call without the
    empty ones, and these hand their states on (h_T over h0 too)."""
    D, lengths = 2, [3, 1, 40, 8, 1, 30, 9]
    N = sum(lengths)
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    g, x, dh = -r(N + 3, D).abs(), r(N + 3, D), r(N + 3, D)
    where = sorted([0, 1, n_seq // 3, n_seq // 3 + 200, n_seq // 2 + 70, n_seq - 2, n_seq - 1])
    counts = torch.zeros(n_seq, dtype=torch.int64, device="cuda")
    counts[where] = torch.tensor(lengths, device="cuda")
    off = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    few_off = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    h0, dh_T = r(n_seq, D), r(n_seq, D)

    def run(n, offsets, h0, dh_T, in_place=False):
        h, dg, dx = (torch.full((N + 3, D), 7.0, device="cuda") for _ in range(3))
        h_T = h0.clone() if in_place else torch.full_like(h0, 7.0)
        dh0, chunks = torch.full_like(h0, 7.0), torch.zeros((2, D), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        head = (N + 3, D, n, offsets, moe.MOE_GLR_MIX, moe.MOE_F32, g, x)
        moe.moe_glr_forward(*head, h_T if in_place else h0, h, h_T, chunks, status)
        moe.moe_glr_backward(*head, h0, chunks, dh, dh_T, dg, dx, dh0, status)
        torch.cuda.synchronize()
        assert int(status) == 0
        return h, dg, dx, h_T, dh0

    want = run(len(lengths), few_off, h0[where].contiguous(), dh_T[where].contiguous())
    for in_place in (False, True):
        got = run(n_seq, off, h0, dh_T, in_place)
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b)
        for a, b, kept in zip(got[3:], want[3:], (h0, dh_T)):
            assert torch.equal(a[where], b)
            a[where] = kept[where]
            assert torch.equal(a, kept)


def test_empty_sequences_without_states_end_in_zeros():
    """h0 NULL: an empty sequence's final state is zero, whoever writes it."""
    for n_seq in (100, 3000):
        off = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
        off[7:] = 2
        g = torch.zeros((2, 40), device="cuda")
        h, h_T = torch.empty_like(g), torch.full((n_seq, 40), 7.0, device="cuda")
        moe.moe_glr_forward(2, 40, n_seq, off, 0, moe.MOE_F32, g, g + 1, None, h, h_T, None)
        assert (h_T[6] == 2).all() and h_T.sum() == 80


@pytest.mark.parametrize("mean", [-0.02, -2.0, -30.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_infinity_stays_in_its_sequence_and_channel(dtype, mean):
    """What the definition makes infinite or NaN is infinite or NaN, the rest has the bits that it
    has without the infinities: mild decays, decays whose product over 64 rows is no fp32 number, and
    decays that are none themselves after three rows."""
    N, D, off = 600, 70, [0, 250, 600]
    gen = torch.Generator().manual_seed(17)
    g = (mean * (0.5 + torch.rand((N, D), generator=gen))).to(dtype).cuda()
    x, dh = (torch.randn((N, D), generator=gen).to(dtype).cuda() for _ in range(2))
    h0, dh_T = (torch.randn((2, D), generator=gen).cuda() for _ in range(2))
    arg = torch.tensor(off, dtype=torch.int32).cuda()
    inf = float("inf")

    def run(x, dh, h0, dh_T):
        h, dg, dx = (torch.empty_like(x) for _ in range(3))
        h_T, dh0 = torch.empty_like(h0), torch.empty_like(h0)
        chunks = torch.empty(((N + 63) // 64, D), device="cuda")
        moe.moe_glr_forward(N, D, 2, arg, 0, CODE[dtype], g, x, h0, h, h_T, chunks)
        moe.moe_glr_backward(N, D, 2, arg, 0, CODE[dtype], g, x, h0, chunks, dh, dh_T, dg, dx, dh0)
        torch.cuda.synchronize()
        return dict(h=h, h_T=h_T, dg=dg, dx=dx, dh0=dh0)

    clean = run(x, dh, h0, dh_T)
    x2, dh2, h02, dh_T2 = x.clone(), dh.clone(), h0.clone(), dh_T.clone()
    h02[0, 3], x2[100, 5], x2[599, 6], x2[260, 7] = inf, -inf, inf, inf  # forward
    dh_T2[1, 10], dh2[400, 12], dh2[0, 13], dh2[249, 14] = -inf, inf, inf, -inf  # backward
    got = run(x2, dh2, h02, dh_T2)
    bad = {n: np.zeros(t.shape, bool) for n, t in got.items()}
    for first, last, c in ((0, 250, 3), (100, 250, 5), (599, 600, 6), (260, 600, 7)):
        bad["h"][first:last, c] = True
        bad["dg"][first + (first != 0):last, c] = True  # a_t lam_t h_{t-1}
        bad["h_T"][int(first >= 250), c] = True
    for first, last, c in ((250, 600, 10), (250, 401, 12), (0, 1, 13), (0, 250, 14)):
        bad["dx"][first:last, c] = True
        bad["dg"][first:last, c] = True
        bad["dh0"][int(first >= 250), c] = True
    for n, t in got.items():
        finite = np.isfinite(f64(t))
        assert not finite[bad[n]].any(), n
        keep = torch.from_numpy(~bad[n]).cuda()
        assert torch.equal(t[keep], clean[n][keep]), n


@pytest.mark.parametrize("which", ["g", "x", "both"])
@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_row_shared_by_all(dtype, D, which):
    """Row stride 0: the forward and the step read one row for all of them."""
    N, slots = 150, 200
    gen = torch.Generator().manual_seed(41)
    whole = dict(g=-torch.rand((N, D), generator=gen), x=torch.randn((N, D), generator=gen))
    i = {n: t.to(dtype).cuda() for n, t in whole.items()}
    for n in ("g", "x") if which == "both" else (which,):
        i[n] = i[n][:1].expand(N, D)
        assert i[n].stride(0) == 0
    h0 = torch.randn((2, D), generator=gen).cuda()
    off = torch.tensor([0, 70, N], dtype=torch.int32).cuda()
    slot = torch.randperm(slots, generator=gen)[:N].to(torch.int32).cuda()
    state = torch.randn((slots, D), generator=gen).cuda()
    old = f64(state)[slot.cpu().numpy()]
    h, hs = (torch.empty((N, D), dtype=dtype, device="cuda") for _ in range(2))
    h_T = torch.empty_like(h0)
    moe.moe_glr_forward(N, D, 2, off, 1, CODE[dtype], i["g"], i["x"], h0, h, h_T, None)
    moe.moe_glr_step(N, D, 1, CODE[dtype], i["g"], i["x"], slot, slots, state, hs)
    torch.cuda.synchronize()
    g, x = f64(i["g"]), f64(i["x"])
    ref, ref_T = SM.gated_recurrence(g, x, [0, 70, N], f64(h0), True)
    E = majorants(g, x, [0, 70, N], f64(h0), True)[1]
    close(h, ref, E, dtype, "h")
    close(h_T, ref_T, E[[69, N - 1]], F32, "h_T")
    rows = list(range(N + 1))
    ref = SM.gated_recurrence(g, x, rows, old, True)[0]
    close(hs, ref, majorants(g, x, rows, old, True)[1], dtype, "step")


def test_no_row_shared_in_an_input_with_a_gradient():
    g = torch.zeros((1, 8), device="cuda").expand(4, 8)
    z = torch.zeros((4, 8), device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_glr_backward(4, 8, 1, None, 0, moe.MOE_F32, g, z, None, z[:1], z, None, g, z + 1, None)


@pytest.mark.parametrize("stride", [4, 8, 1 << 40])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_stride_of_a_single_row_means_nothing(dtype, stride):
    """One row: whatever its tensor says of the next one, forward and backward."""
    D = 256
    gen = torch.Generator().manual_seed(43)
    g, x, dh = (torch.randn((1, D), generator=gen).to(dtype).cuda() for _ in range(3))
    g = -g.abs()
    one = lambda t: t.as_strided((1, D), (stride, 1))  # noqa: E731
    h, dg, dx = (torch.empty((1, D), dtype=dtype, device="cuda") for _ in range(3))
    chunks = torch.empty((1, D), device="cuda")
    moe.moe_glr_forward(1, D, 1, None, 0, CODE[dtype], one(g), one(x), None, h, None, chunks)
    moe.moe_glr_backward(1, D, 1, None, 0, CODE[dtype], one(g), one(x), None, chunks, dh, None,
                         one(dg), one(dx), None)
    torch.cuda.synchronize()
    assert torch.equal(h, x) and torch.equal(dx, dh) and (dg == 0).all()
