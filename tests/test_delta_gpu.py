"""The gated delta memory on the GPU against its 64-bit form (delta_ref): forward, gradients and decoding, every
aggregation, element type and head dimension, ragged and one-token lengths.

Tolerances, relative to the largest reference value of an output:
  fp32   1e-4, the forward's: sums of at most a few thousand products at 2^-24 each, which add up like their root
         (2^-24 * sqrt(1000 * 128) = 2e-5), times five for the chain of a segment's tokens.
  bf16   1e-2, the forward's: the rounding of the result is off by up to 2^-8 = 3.9e-3 of itself, and the operands
         that are rounded on the way (2^-8 each at most) add up like their root over the terms of a sum.
  states from bf16 inputs 1e-4: the inputs are exact in fp32 and the memory is held in it.
"""
import numpy as np
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, MEAN, RESIDUAL, SOUP, SSC, backward, forward, make_delta_inputs

pytestmark = pytest.mark.gpu

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


SHAPES = [  # (d, C, L, dtype): whole, ragged and one-token segments, lengths next to the 64-token chunks
    (16, 16, 50, "f32"), (32, 37, 130, "f32"), (64, 64, 192, "f32"), (128, 100, 230, "f32"),
    (16, 20, 61, "bf16"), (32, 64, 129, "bf16"),
    (64, 64, 192, "bf16"), (64, 65, 200, "bf16"), (64, 128, 512, "bf16"), (64, 1, 5, "bf16"),
    (128, 128, 384, "bf16"), (128, 63, 190, "bf16"), (128, 130, 300, "bf16"), (128, 256, 512, "bf16"), (64, 256, 768, "bf16"),
]
UNCUT = [(16, 1, "f32"), (64, 63, "bf16"), (64, 300, "bf16"), (128, 1, "bf16"), (128, 64, "bf16"), (128, 257, "bf16"), (128, 200, "f32"), (64, 129, "f32")]


@pytest.mark.parametrize("mode,topk", [(RESIDUAL, 0), (GRM, 0), (SOUP, 0), (SSC, 1), (MEAN, 0)])
@pytest.mark.parametrize("d,C,L,dtype", SHAPES)
def test_forward(d, C, L, dtype, mode, topk):
    x = make_delta_inputs(2, 2, L, d, C, d + C + L, dtype)
    y, st = forward(*x, C, mode, topk)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, mode, topk)
    assert mcl.mc_check_device() == mcl.MC_OK
    assert rel(gy, y) <= TOL[dtype]
    assert rel(gst, st) <= STATE_TOL
    again, none = mcl.mc_forward_delta(*cuda(x), C, mode, topk, want_states=False)
    assert none is None and rel(again, y) <= TOL[dtype]
    if dtype == "f32" or d < 64:  # the tensor-core kernels hold the states to more terms when they are returned
        assert torch.equal(again, gy)


@pytest.mark.parametrize("d,L,dtype", UNCUT)
def test_forward_of_one_memory(d, L, dtype):
    x = make_delta_inputs(1, 3, L, d, L, d + L, dtype)
    y, st = forward(*x, L, RESIDUAL)
    q, k, v, u, la, be = cuda(x)
    gy, gst = mcl.mc_forward_delta(q, k, v, None, la, be, L + 5, RESIDUAL)
    assert rel(gy, y) <= TOL[dtype] and rel(gst, st) <= STATE_TOL
    assert torch.equal(mcl.mc_forward_delta(q, k, v, u, la, be, L, GRM)[0], gy)


def test_lengths_past_many_chunks():
    x = make_delta_inputs(1, 1, 2500, 64, 2500, 5, "bf16", decay=0.002)
    y, st = forward(*x, 2500, RESIDUAL)
    gy, gst = mcl.mc_forward_delta(*cuda(x), 2500, RESIDUAL)
    assert rel(gy, y) <= TOL["bf16"] and rel(gst, st) <= STATE_TOL


@pytest.mark.parametrize("dtype,d,L,C", [("f32", 32, 150, 70), ("bf16", 64, 150, 70), ("bf16", 128, 150, 70), ("bf16", 64, 256, 128),
                                         ("bf16", 128, 256, 128)])
def test_the_ends_of_the_gates(dtype, d, L, C):
    """No decay, a full reset, no write, and writes past the value (beta = 2), next to one another."""
    q, k, v, u, la, be = make_delta_inputs(1, 2, L, d, C, 9, dtype)
    la[:, :, ::3] = 0.0
    la[:, :, 10::17] = -80.0
    la[:, :, 75] = -float("inf")
    la[:, :, C] = -float("inf")  # a segment's first token
    be[:, :, ::5] = 0.0
    be[:, :, 3::7] = 2.0
    x = [q, k, v, u, la, be]
    floor = [q, k, v, u, la.double().clamp_min(-60.0), be]
    y, st = forward(*floor, C, GRM)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, GRM)
    assert rel(gy, y) <= TOL[dtype] and rel(gst, st) <= STATE_TOL
    dy = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(q.dtype)
    for g, w in zip(mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, GRM), backward(*floor, dy, C, GRM)):
        assert torch.isfinite(g).all() and rel(g, w) <= TOL[dtype]


@pytest.mark.parametrize("mode,topk", [(RESIDUAL, 0), (GRM, 0), (SSC, 1), (MEAN, 0)])
@pytest.mark.parametrize("d,C,L,dtype", SHAPES)
def test_backward(d, C, L, dtype, mode, topk):
    x = make_delta_inputs(1, 2, L, d, C, d + C + L + 1, dtype)
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(L)).to(x[0].dtype)
    want = backward(*x, dy, C, mode, topk)
    got = mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, mode, topk)
    assert mcl.mc_check_device() == mcl.MC_OK
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, want):
        if g is None:
            assert mode in (RESIDUAL, MEAN) and not w.any()
        else:
            assert rel(g, w) <= TOL[dtype], name


@pytest.mark.parametrize("d,L,dtype", UNCUT)
def test_backward_of_one_memory(d, L, dtype):
    x = make_delta_inputs(1, 3, L, d, L, d + L, dtype)
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(L)).to(x[0].dtype)
    want = backward(*x, dy, L, RESIDUAL)
    q, k, v, u, la, be = cuda(x)
    got = mcl.mc_backward_delta(q, k, v, None, la, be, dy.cuda(), L, RESIDUAL)
    assert got[3] is None
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, want):
        if g is not None:
            assert rel(g, w) <= TOL[dtype], name
    du = torch.full_like(q, 7.0)  # a single memory has nothing to weigh
    mcl.mc_backward_delta(q, k, v, u, la, be, dy.cuda(), L, GRM, du=du)
    assert not du.any()


def test_long_decays_keep_their_gradient():
    """The decay's gradient is a difference of running sums; over many chunks it stays as exact as the others."""
    L, d = 1500, 64
    x = make_delta_inputs(1, 1, L, d, L, 11, "bf16", decay=0.05)
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(2)).to(x[0].dtype)
    want = backward(*x, dy, L, RESIDUAL)
    got = mcl.mc_backward_delta(*cuda(x), dy.cuda(), L, RESIDUAL)
    for n in (0, 1, 2, 4, 5):
        assert rel(got[n], want[n]) <= TOL["bf16"], n


def test_autograd():
    x = cuda(make_delta_inputs(1, 2, 100, 64, 40, 3, "bf16"))
    leaf = [t.clone().requires_grad_() for t in x]
    y = mcl.DeltaMemoryCaching.apply(*leaf, 40, GRM, 0)
    dy = torch.randn_like(y)
    y.backward(dy)
    for t, w in zip(leaf, mcl.mc_backward_delta(*x, dy, 40, GRM)):
        assert rel(t.grad, w.cpu()) <= TOL["bf16"]
    leaf = [t.clone().requires_grad_() for t in x]
    mcl.DeltaMemoryCaching.apply(*leaf, 100, MEAN, 0).backward(dy)
    assert not leaf[3].grad.any()
    leaf[3] = None
    mcl.DeltaMemoryCaching.apply(*leaf, 100, MEAN, 0).backward(dy)


@pytest.mark.parametrize("mode,topk", [(RESIDUAL, 0), (GRM, 0), (SOUP, 0), (SSC, 2), (MEAN, 0)])
@pytest.mark.parametrize("d,C,L,dtype", [(16, 7, 30, "f32"), (32, 10, 45, "bf16"), (64, 16, 70, "bf16"), (128, 12, 50, "f32"), (128, 3, 190, "bf16")])
def test_decode_reproduces_the_forward(d, C, L, dtype, mode, topk):
    x = make_delta_inputs(2, 2, L, d, C, 21, dtype)
    y, st = forward(*x, C, mode, topk)
    xd = cuda(x)
    cache = mcl.DecodeCache(2, 2, d, C, min(64, -(-L // C)))
    for t in cache.states, cache.kbar, cache.online, cache.ksum:
        t.fill_(float("nan"))  # contents are ignored at t = 0
    got = torch.stack([mcl.mc_decode_step_delta(cache, *(t[:, :, j].contiguous() for t in xd), mode, topk) for j in range(L)], 2)
    assert rel(got, y) <= TOL[dtype]
    done = L // C
    assert rel(cache.states[:, :, :done], st[:, :, :done]) <= STATE_TOL
    with pytest.raises(mcl.MCError) as e:
        cache.t = cache.n_max * C
        mcl.mc_decode_step_delta(cache, *(t[:, :, 0].contiguous() for t in xd), mode, topk)
    assert e.value.status == mcl.MC_ERR_SHAPE


def test_prefill_then_decode():
    """A prefill's states hand over to decoding: the steps continue the forward."""
    B, H, L, P, d, C = 1, 2, 200, 150, 64, 32
    x = make_delta_inputs(B, H, L, d, C, 31, "bf16")
    y, _ = forward(*x, C, GRM)
    xd = cuda(x)
    head = [t[:, :, :P].contiguous() for t in xd]
    _, st = mcl.mc_forward_delta(*head, C, GRM)
    cache = mcl.EvictingCache(B, H, d, C, 16)
    mcl.mc_cache_compact(cache, head[1], head[3], st, GRM)
    got = []
    for j in range(P, L):
        tok = [t[:, :, j].contiguous() for t in xd]
        got.append(mcl.mc_decode_step_evict(cache, *tok[:4], GRM, log_alpha=tok[4], beta=tok[5]))
    assert rel(torch.stack(got, 2), y[:, :, P:]) <= TOL["bf16"]


def test_streams_and_graphs():
    x = cuda(make_delta_inputs(1, 2, 300, 64, 100, 41, "bf16"))
    dy = torch.randn_like(x[0])
    want = mcl.mc_forward_delta(*x, 100, GRM)
    grads = mcl.mc_backward_delta(*x, dy, 100, GRM)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mcl.mc_forward_delta(*x, 100, GRM)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for _ in range(2):  # two captured graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = mcl.mc_forward_delta(*x, 100, GRM) + mcl.mc_backward_delta(*x, dy, 100, GRM)
        graphs.append((g, out))
    for _ in range(2):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            for a, b in zip(out[2:], grads):
                assert rel(a, b.cpu()) <= TOL["bf16"]


def test_nothing_is_written_behind_the_outputs():
    B, H, L, d, C = 1, 2, 77, 64, 30
    x = cuda(make_delta_inputs(B, H, L, d, C, 51, "bf16"))
    n = B * H * L * d
    buf = torch.full((2 * n,), 3.0, dtype=torch.bfloat16, device="cuda")
    mcl.mc_forward_delta(*x, C, GRM, y=buf[:n].view(B, H, L, d))
    assert (buf[n:] == 3.0).all()
    big = [torch.full((2 * t.numel(),), 3.0, dtype=t.dtype, device="cuda") for t in x]
    outs = {name: b[:t.numel()].view(t.shape) for name, b, t in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), big, x)}
    mcl.mc_backward_delta(*x, torch.ones_like(x[0]), C, GRM, **outs)
    for b, t in zip(big, x):
        assert (b[t.numel():] == 3.0).all()


@pytest.mark.parametrize("d,C,L", [(64, 30, 310), (128, 70, 350), (128, 128, 640), (64, 128, 1280)])
def test_many_heads_and_segments(d, C, L):
    """Enough walkers to fill the card: one warp per 16 rows instead of two."""
    x = make_delta_inputs(2, 8, L, d, C, 61, "bf16")
    y, st = forward(*x, C, GRM)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, GRM)
    assert rel(gy, y) <= TOL["bf16"] and rel(gst, st) <= STATE_TOL
    assert rel(mcl.mc_forward_delta(*cuda(x), C, GRM, want_states=False)[0], y) <= TOL["bf16"]
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(8)).to(x[0].dtype)
    got = mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, GRM)
    assert mcl.mc_check_device() == mcl.MC_OK
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, backward(*x, dy, C, GRM)):
        assert rel(g, w) <= TOL["bf16"], name


@pytest.mark.parametrize("beta", [1.0, 1.9])
@pytest.mark.parametrize("d,dtype", [(32, "f32"), (64, "bf16"), (128, "bf16")])
def test_keys_that_resemble_each_other(d, dtype, beta):
    """Neighbouring keys all but parallel: the inverse within a chunk is far from the identity, and every write undoes
    the one before, so the values e_j beta_j that a chunk writes are of the size of the result and cancel.

    States from bf16 inputs: an operand of two bf16 terms is off by 2^-17 of itself, and the 64 products of a chunk's
    sum by the root of that, 8 * 2^-17 = 6e-5 of the largest; the memory forgets a write by |1 - beta| per token, so at
    beta = 1.9 the errors of 1 / (1 - 0.9) = 10 tokens stand together: 6e-4, and at beta = 1 of one.  Over two chunks and
    the decay of a maximum over 2 d^2 entries (four standard deviations), 2.5e-4 and 2.5e-3.
    y with cached segments: the readout's tensor-core kernels round the written values and their weights to bf16, 2^-9 in
    the mean, and a token's read has 128 products of a chunk of which each counts: 2^-9 * sqrt(2 * 128) = 3e-2, times
    four standard deviations over values of which the largest is at four, too.  One memory is read in two terms: 1e-2.
    Gradients pass through bf16 e, w and states the same way: chunks of 64, three roundings, 2^-9 * sqrt(3 * 64) = 2.7e-2,
    times |beta| of the write that they go through twice."""
    L, C = 260, 128
    q, k, v, u, la, be = make_delta_inputs(1, 2, L, d, C, 71, dtype, decay=0.001)
    k = k.float() * 0.05 + k[:, :, :1].float()
    k = (k / k.norm(dim=-1, keepdim=True)).to(q.dtype)
    be = torch.full_like(be, beta)
    x = [q, k, v, u, la, be]
    dy = torch.randn(q.shape, generator=torch.Generator().manual_seed(9)).to(q.dtype)
    y1, st1 = forward(*x, L, RESIDUAL)
    gy1, gst1 = mcl.mc_forward_delta(*cuda(x), L, RESIDUAL)
    y, st = forward(*x, C, GRM)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, GRM)
    b16 = dtype == "bf16"
    state_tol = STATE_TOL if not b16 else 2.5e-4 if beta == 1.0 else 2.5e-3
    print("states", rel(gst, st), rel(gst1, st1), "y", rel(gy, y), rel(gy1, y1))
    assert rel(gy1, y1) <= TOL[dtype] and rel(gst1, st1) <= state_tol
    assert rel(gst, st) <= state_tol and rel(gy, y) <= (3e-2 if b16 else TOL[dtype])
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, GRM),
                          backward(*x, dy, C, GRM)):
        print(name, rel(g, w))
        assert rel(g, w) <= (2.7e-2 * max(1.0, beta) ** 2 if b16 else TOL[dtype]), name


def test_offsets_past_32_bits():
    """More than 2^31 elements in every tensor and in the chunk states: copies of one head, the last as the first."""
    if torch.cuda.mem_get_info()[0] < 170e9:
        pytest.skip("needs 170 GB")
    BH, L, d, C = 33000, 1024, 64, 128
    assert BH * L * d > 2**31 and BH * (L // 64) * d * d > 2**31
    one = make_delta_inputs(1, 1, L, d, C, 81, "bf16")
    dy1 = torch.randn(one[0].shape, generator=torch.Generator().manual_seed(10)).to(one[0].dtype)
    y, st = forward(*one, C, GRM)
    want = backward(*one, dy1, C, GRM)
    x = [t.cuda().expand(1, BH, *t.shape[2:]).contiguous() for t in one]
    dy = dy1.cuda().expand(1, BH, L, d).contiguous()
    gy, gst = mcl.mc_forward_delta(*x, C, GRM)
    for h in (0, BH - 1):
        assert rel(gy[:, h], y[:, 0]) <= TOL["bf16"] and rel(gst[:, h], st[:, 0]) <= STATE_TOL
    assert torch.equal(gy[:, 0], gy[:, -1]) and torch.equal(gst[:, 0], gst[:, -1])
    del gy, gst
    got = mcl.mc_backward_delta(*x, dy, C, GRM)
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, want):
        assert rel(g[:, 0], w[:, 0]) <= TOL["bf16"] and rel(g[:, -1], w[:, 0]) <= TOL["bf16"], name
    del x, dy, got, g
    mcl.mc_trim_scratch()
    torch.cuda.empty_cache()


def test_second_gradients_are_refused():
    x = [t.requires_grad_() for t in cuda(make_delta_inputs(1, 1, 20, 16, 10, 4, "f32"))]
    y = mcl.DeltaMemoryCaching.apply(*x, 10, GRM, 0)
    dq, = torch.autograd.grad(y.square().sum(), x[0], create_graph=True)
    with pytest.raises(RuntimeError):
        dq.sum().backward()


@pytest.mark.parametrize("d,dtype", [(32, "f32"), (64, "bf16"), (128, "bf16")])
def test_neighbours_do_not_leak(d, dtype):
    """NaN in another segment or another head: tiles of 64 tokens reach over a segment's end and must not use what is there."""
    L, C = 290, 100
    clean = cuda(make_delta_inputs(1, 2, L, d, C, 95, dtype))
    bad = [t.clone() for t in clean]
    for t in bad:
        t[:, :, C:] = float("nan")
    for mode in (RESIDUAL, GRM):
        y, st = mcl.mc_forward_delta(*clean, C, mode)
        yb, stb = mcl.mc_forward_delta(*bad, C, mode)
        assert torch.equal(yb[:, :, :C], y[:, :, :C]) and torch.equal(stb[:, :, 0], st[:, :, 0])
        assert torch.isnan(yb[:, :, C:]).all()
    bad = [t.clone() for t in clean]
    for t in bad:
        t[:, 1] = float("nan")
    dy = torch.randn(clean[0].shape, generator=torch.Generator().manual_seed(11)).to(clean[0])
    dyb = dy.clone()
    dyb[:, 1] = float("nan")
    for C in (100, 70, L):
        assert torch.equal(mcl.mc_forward_delta(*bad, C, GRM)[0][:, 0], mcl.mc_forward_delta(*clean, C, GRM)[0][:, 0])
        want, got = mcl.mc_backward_delta(*clean, dy, C, GRM), mcl.mc_backward_delta(*bad, dyb, C, GRM)
        for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, want):
            assert rel(g[:, 0], w[:, 0].cpu()) <= TOL[dtype] / 10, name


@pytest.mark.parametrize("d,C,L,dtype,mode,topk", [(16, 1, 300, "f32", GRM, 0), (64, 1, 300, "bf16", GRM, 0), (64, 2, 301, "bf16", SSC, 3),
                                                   (64, 128, 2560, "bf16", SSC, 17), (128, 128, 2560, "bf16", SSC, 1)])
def test_many_short_segments_and_wide_routers(d, C, L, dtype, mode, topk):
    x = make_delta_inputs(1, 1, L, d, C, 97, dtype)
    y, st = forward(*x, C, mode, topk)
    gy, gst = mcl.mc_forward_delta(*cuda(x), C, mode, topk)
    assert rel(gy, y) <= TOL[dtype] and rel(gst, st) <= STATE_TOL
    dy = torch.randn(x[0].shape, generator=torch.Generator().manual_seed(12)).to(x[0].dtype)
    got = mcl.mc_backward_delta(*cuda(x), dy.cuda(), C, mode, topk)
    assert mcl.mc_check_device() == mcl.MC_OK
    for name, g, w in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got, backward(*x, dy, C, mode, topk)):
        assert rel(g, w) <= TOL[dtype], name
