"""The gated delta memory's tensor-core kernels when a bounded wait gives up: the call is reported, nothing hangs, and the
next call is right.  The waits give up on request (mc_selftest_delta_give_up); the copies they wait for are good ones."""
import ctypes

import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, RESIDUAL, make_delta_inputs

pytestmark = pytest.mark.gpu

TILES, LATE, END = 1, 2, 4


@pytest.fixture(scope="module")
def give_up():
    from memory_caching_linear_gb300 import build
    build.build()
    lib = mcl.load_library()
    lib.mc_selftest_delta_give_up.argtypes, lib.mc_selftest_delta_give_up.restype = [ctypes.c_int], ctypes.c_int
    assert lib.mc_selftest_delta_give_up(8) == mcl.MC_ERR_MODE
    yield lib.mc_selftest_delta_give_up
    lib.mc_selftest_delta_give_up(0)


def inputs(H, L, d, C):
    """Two heads, the others as copies: enough heads that a warp takes whole rows (its records come late)."""
    x = [t.cuda() for t in make_delta_inputs(1, 2, L, d, C, H + L + d, "bf16")]
    return [t.repeat(1, H // 2, *[1] * (t.dim() - 2)).contiguous() for t in x]


def forward(x, C, mode):
    return [t for t in mcl.mc_forward_delta(*x, C, mode)]


def backward(x, C, mode):
    g = torch.Generator("cuda").manual_seed(1)
    return [t for t in mcl.mc_backward_delta(*x, torch.randn(x[0].shape, device="cuda", generator=g).to(x[0].dtype), C, mode) if t is not None]


# (heads, L, d, C): few heads (two warps to a row) and many; one chunk, whose wait is the last one, and several
SHAPES = [(2, 64, 64, 64), (2, 300, 128, 300), (200, 64, 64, 64), (100, 50, 128, 50), (200, 200, 64, 200), (100, 256, 128, 128)]


@pytest.mark.parametrize("H,L,d,C", SHAPES)
@pytest.mark.parametrize("call,waits", [(forward, TILES), (forward, LATE), (backward, TILES), (backward, LATE), (backward, END)])
def test_waits_that_give_up_are_reported(give_up, call, waits, H, L, d, C):
    x = inputs(H, L, d, C)
    mode = RESIDUAL if C >= L else GRM
    want = call(x, C, mode)
    assert mcl.mc_check_device() == mcl.MC_OK
    if call is forward and waits == LATE and (C < L or H == 2):
        waits |= TILES  # (these walks have no late wait)
    assert give_up(waits) == mcl.MC_OK
    call(x, C, mode)
    assert give_up(0) == mcl.MC_OK
    assert mcl.mc_check_device() == mcl.MC_ERR_DEVICE_TIMEOUT
    assert mcl.mc_check_device() == mcl.MC_OK  # reported once
    got = call(x, C, mode)
    assert mcl.mc_check_device() == mcl.MC_OK
    for a, b in zip(got, want):
        scale = float(b.abs().max())
        assert float((a.double() - b.double()).abs().max()) <= 1e-3 * scale  # (the pooled keys' gradient is summed by atomics)
