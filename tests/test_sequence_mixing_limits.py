"""CPU checks of the limits of the operators beside the gated delta rule: sizes and addresses that a
call refuses before anything reaches a GPU."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

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


FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
INVALID, UNSUPPORTED = 1, 2


def gdr_step(B=4, H=2, dk=64, dv=64, q=FAKE, k=FAKE, v=FAKE, beta=FAKE, g=FAKE, slot=FAKE,
             n_slots=1 << 24, S=FAKE, o=FAKE, status=None):
    return moe.lib().moe_gdr_step(B, H, dk, dv, q, k, v, beta, g, slot, n_slots, 0.1, S, o, status,
                                  None)


def test_steps_refuse_batches_whose_slots_take_too_long_to_compare():
    """Every request looks for its slot among those before it, which grows with the square of the
    batch."""
    assert gdr_step(B=65536, H=1) == UNSUPPORTED
    assert gdr_step(B=1 << 24, H=1) == UNSUPPORTED
    assert gdr_step(B=1 << 13, H=(1 << 11) + 1, slot=None) == UNSUPPORTED
    assert moe.lib().moe_glr_step(65536, 8, 0, 0, FAKE, 8, FAKE, 8, FAKE, 1 << 24, FAKE, FAKE, None,
                                  None) == UNSUPPORTED


def test_limits_of_the_steps_are_documented():
    with open(os.path.join(B.ROOT, "include", "linear_attention.h")) as f:
        text = " ".join(f.read().split())
    assert "B * H up to 2^24" in text and "B up to 65535" in text


CHOICE = r"""
#include "cluster_room.h"
extern "C" void choose(const int* fits, int strips, int tiles, int n_seq, int* out) {
  const moe::ClusterRoom room = moe::ask_room([&](int c, int* n) {
    *n = fits[c];
    return fits[c] >= 0;  // negative: the driver refuses the size
  });
  const moe::ClusterChoice c = moe::choose_clusters(room, strips, tiles, n_seq);
  out[0] = c.cluster;
  out[1] = c.parts;
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    at = tmp_path_factory.mktemp("choice")
    (at / "choice.cpp").write_text(CHOICE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, str(at / "choice.cpp"),
                    "-o", str(at / "choice.so")], check=True)
    f = ctypes.CDLL(str(at / "choice.so")).choose

    def call(fits, strips, tiles, n_seq):
        out = (ctypes.c_int * 2)()
        f((ctypes.c_int * 17)(*fits), strips, tiles, n_seq, out)
        return tuple(out)

    return call


FITS = [0] + [304 // c for c in range(1, 17)]  # two blocks to each of 152 SMs, nothing lost to size


def test_clusters_are_as_large_as_fit(choose):
    assert choose(FITS, 36, 1000, 1) == (8, 1)        # 36 strips: 38 clusters of 8 fit, 33 of 9
    assert choose(FITS, 32, 1000, 1) == (9, 1)        # 32 strips: one block more for each
    assert choose(FITS, 40, 1000, 1) == (7, 1)        # 38 clusters of 8 do not hold 40 strips
    assert choose(FITS, 1, 1000, 1) == (16, 1)        # few channels: more blocks to work
    assert choose(FITS, 1, 1000, 100) == (8, 38)      # with many sequences parts do that
    assert choose(FITS, 1, 3, 1) == (3, 1)            # no more blocks than tiles
    assert choose(FITS, 400, 1000, 5) == (1, 1)       # more strips than places


def test_cluster_sizes_that_the_driver_refuses_are_left_out(choose):
    """A size that cannot be launched here costs that size, not every call."""
    few = [n if c <= 8 else -1 for c, n in enumerate(FITS)]
    assert choose(few, 1, 1000, 1) == (8, 1)
    holes = [-1 if c in (8, 16, 15) else n for c, n in enumerate(FITS)]
    assert choose(holes, 36, 1000, 1) == (7, 1)
    assert choose(holes, 32, 1000, 1) == (9, 1)
    assert choose(holes, 1, 1000, 1) == (14, 1)
    none = [-1] * 17
    assert choose(none, 32, 1000, 10) == (1, 1)


def glr(backward=False, **over):
    a = dict(N=8, D=5, n_seq=2, off=FAKE, mode=0, dtype=0, g=FAKE, ld_g=5, x=FAKE, ld_x=5, h0=FAKE,
             h=FAKE, h_T=FAKE, chunks=FAKE, dh=FAKE, dh_T=FAKE, dg=FAKE, dx=FAKE, dh0=FAKE,
             status=FAKE)
    a.update(over)
    names = ["N", "D", "n_seq", "off", "mode", "dtype", "g", "ld_g", "x", "ld_x", "h0"]
    names += ["chunks", "dh", "dh_T", "dg", "dx", "dh0"] if backward else ["h", "h_T", "chunks"]
    call = moe.lib().moe_glr_backward if backward else moe.lib().moe_glr_forward
    return call(*[a[n] for n in names + ["status"]], None)


def test_addresses_off_their_types_boundary_are_refused():
    """A kernel would fault on them."""
    for off in (1, 2, 3):
        at = FAKE + off
        for n in ("off", "h0", "h_T", "chunks", "status"):
            assert glr(**{n: at}) == UNSUPPORTED, n
        for n in ("off", "h0", "chunks", "dh_T", "dh0", "status"):
            assert glr(backward=True, **{n: at}) == UNSUPPORTED, n
        for n in ("beta", "g", "slot", "status"):
            assert gdr_step(**{n: at}) == UNSUPPORTED, n
        for slot, state, status in ((at, FAKE, None), (FAKE, at, None), (FAKE, FAKE, at)):
            assert moe.lib().moe_glr_step(4, 5, 0, 0, FAKE, 5, FAKE, 5, slot, 4, state, FAKE, status,
                                          None) == UNSUPPORTED
    rows = moe.moe_qk_rows(x=FAKE, x_token_stride=256, x_head_stride=64, y=FAKE, y_token_stride=256,
                           y_head_stride=64, heads=4)
    grads = moe.moe_qk_grads(x=FAKE, x_token_stride=256, x_head_stride=64, dy=FAKE,
                             dy_token_stride=256, dy_head_stride=64, dx=FAKE, dx_token_stride=256,
                             dx_head_stride=64, heads=4)
    for pos, freq in ((FAKE + 2, FAKE), (FAKE, FAKE + 4)):
        assert moe.lib().moe_qk_norm_rope(8, 64, 64, 0, 0, 1e-6, pos, freq, ctypes.byref(rows), None,
                                          None) == UNSUPPORTED
        assert moe.lib().moe_qk_norm_rope_backward(8, 64, 64, 0, 0, 1, 1e-6, pos, freq,
                                                   ctypes.byref(grads), None, None, 0,
                                                   None) == UNSUPPORTED


@pytest.mark.parametrize("dtype", [7, -1, None])
def test_binding_refuses_types_that_it_does_not_know(dtype):
    """With the error that it raises for every other argument that is not what a call takes."""
    z, x = torch.zeros((4, 8)), torch.zeros((4, 2, 64))
    pos, freq = torch.arange(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    q, f = dict(x=x, y=x, dy=x, dx=x), moe.MOE_F32
    calls = [lambda: moe.moe_glr_forward(4, 8, 1, None, 0, dtype, z, z, None, z, None, None),
             lambda: moe.moe_glr_backward(4, 8, 1, None, 0, dtype, z, z, None, z[:1], z, None, z, z,
                                          None),
             lambda: moe.moe_glr_step(4, 8, 0, dtype, z, z, None, 4, z, z),
             lambda: moe.moe_qk_norm_rope(4, 64, 64, False, dtype, 1e-6, pos, freq, q, None),
             lambda: moe.moe_qk_norm_rope_backward(4, 64, 64, False, dtype, f, 1e-6, pos, freq, q,
                                                   None, None),
             lambda: moe.moe_qk_norm_rope_backward(4, 64, 64, False, f, dtype, 1e-6, pos, freq, q,
                                                   None, None)]
    for call in calls:
        with pytest.raises(ValueError, match="MOE_BF16 or MOE_F32"):
            call()
