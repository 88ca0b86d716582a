"""How exact the gated delta memory is where its gates or keys make that hard, against the 64-bit form (delta_ref).

Errors are relative to the largest reference value of an output, as in test_delta_gpu.py, and so are the tolerances that
these tests share with it: 1e-4 for fp32 results and for states, 1e-2 for bf16 results."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, MEAN, RESIDUAL, SSC, backward, forward, make_delta_inputs

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "du", "dlog_alpha", "dbeta")
TOL = {"f32": 1e-4, "bf16": 1e-2}
STATE_TOL = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from memory_caching_linear_gb300 import build
    build.build()
    mcl.load_library()


def rel(got, ref):
    ref = ref.double()
    scale = float(ref.abs().max())
    return float((got.double().cpu() - ref).abs().max()) / (scale if scale > 0 else 1.0)


def cuda(xs):
    return [x.cuda() if x is not None else None for x in xs]


def after_resets(H, L, d, C, dtype, resets):
    """Every chunk of 64 tokens starts with so many full resets and goes on with ordinary decays; the ends of the segments
    lie in such a stretch."""
    x = make_delta_inputs(1, H, L, d, C, d + resets, dtype, decay=0.05)
    for s in range(0, L, 64):
        x[4][:, :, s:s + resets] = -float("inf")
    return x, [*x[:4], x[4].double().clamp_min(-60.0), x[5]]


@pytest.mark.parametrize("resets", [48, 56, 60])
@pytest.mark.parametrize("d,C,L", [(64, 128, 256), (64, 64, 64), (128, 128, 128), (128, 192, 384)])
def test_states_after_many_resets(d, C, L, resets):
    """The decay between two neighbouring tokens is one number whatever came before them."""
    x, floor = after_resets(4, L, d, C, "bf16", resets)
    y, st = forward(*floor, C, GRM)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, GRM)
    assert rel(gst, st) <= STATE_TOL and rel(gy, y) <= TOL["bf16"]


@pytest.mark.parametrize("resets", [40, 60])
@pytest.mark.parametrize("d,C,L,mode", [(16, 64, 128, GRM), (32, 64, 64, RESIDUAL), (64, 128, 256, GRM), (128, 64, 64, RESIDUAL)])
def test_fp32_gradients_after_many_resets(d, C, L, mode, resets):
    x, floor = after_resets(2, L, d, C, "f32", resets)
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(3))
    for name, g, w in zip(NAMES, mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, mode), backward(*floor, dy, C, mode)):
        if g is not None:
            assert rel(g, w) <= TOL["f32"], name


def resembling(L, d, spread, beta, seed=71):
    """Neighbouring keys that share one direction: every write undoes the one before, so what a chunk writes is of the size of
    the result and cancels."""
    q, k, v, u, la, be = make_delta_inputs(1, 2, L, d, 128, seed, "bf16", decay=0.001)
    k = k.float() * spread + k[:, :, :1].float()
    return [q, (k / k.norm(dim=-1, keepdim=True)).to(q.dtype), v, u, la, torch.full_like(be, beta)]


@pytest.mark.parametrize("mode,topk", [(RESIDUAL, 0), (GRM, 0), (SSC, 1), (MEAN, 0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread,beta", [(0.05, 1.0), (0.05, 1.9), (0.3, 1.9)])
@pytest.mark.parametrize("C,L", [(128, 384), (130, 384), (192, 384), (384, 384), (128, 380)])
def test_reads_of_resembling_keys(C, L, spread, beta, d, mode, topk):
    """y is as exact for one segment length as for another: whatever kernels read the cached memories, the online read is
    formed in two bf16 terms, 2^-17 of the terms that cancel, and what remains of the 1e-2 are roundings of results."""
    x = resembling(L, d, spread, beta)
    y, _ = forward(*x, C, mode, topk)
    assert rel(mcl.mc_forward_delta(*cuda(x), C, mode, topk)[0], y) <= TOL["bf16"]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread,beta", [(0.05, 1.0), (0.05, 1.9), (0.3, 1.9)])
@pytest.mark.parametrize("C,L", [(128, 256), (130, 260), (192, 256), (256, 256)])
def test_gradients_of_resembling_keys(C, L, spread, beta, d):
    """Sums over pairs of tokens cancel here; formed in two bf16 terms, 2^-17, as is the adjoint's read, they leave the 1e-2 of
    bf16 results (in one term dq and dbeta were 5e-2 off).  dlog_alpha is a difference of reads and writes: its bound is that
    of test_keys_that_resemble_each_other."""
    x = resembling(L, d, spread, beta)
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(9)).to(x[0].dtype)
    tol = {"dlog_alpha": 2.7e-2 * max(1.0, beta) ** 2}
    for name, g, w in zip(NAMES, mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, GRM), backward(*x, dy, C, GRM)):
        assert rel(g, w) <= tol.get(name, TOL["bf16"]), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("C,L,mode", [(128, 256, GRM), (128, 256, RESIDUAL), (130, 260, GRM), (256, 256, GRM)])
def test_gradients_in_the_mean(C, L, mode, d):
    """In the 2-norm a rounding to bf16 is 1.7e-3 (2^-8 / sqrt(3) times the mean of a value over its power of two, 0.74).  A
    gradient has its own, that of the state or adjoint it reads, and, behind gates, theirs: 1.7e-3 * sqrt(3) = 2.9e-3."""
    x = make_delta_inputs(2, 3, L, d, C, 7 + d, "bf16")
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(9)).to(x[0].dtype)
    for name, g, w in zip(NAMES, mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, mode), backward(*x, dy, C, mode)):
        if g is not None and name != "dlog_alpha" and w.any():
            assert float((g.double().cpu() - w).norm() / w.norm()) <= 2.9e-3, name


@pytest.mark.parametrize("d,C,L", [(16, 20, 61), (32, 64, 129), (64, 64, 192), (64, 128, 512), (128, 130, 300), (128, 128, 384), (128, 257, 257)])
@pytest.mark.parametrize("mode,topk", [(RESIDUAL, 0), (GRM, 0), (SSC, 1)])
def test_states_or_not_the_same_y(d, C, L, mode, topk):
    """A call that returns no states, as the autograd function makes it, forms the same y, bit for bit."""
    x = cuda(make_delta_inputs(2, 2, L, d, C, d + C, "bf16"))
    y, st = mcl.mc_forward_delta(*x, C, mode, topk)
    again, none = mcl.mc_forward_delta(*x, C, mode, topk, want_states=False)
    assert none is None and torch.equal(again, y)
