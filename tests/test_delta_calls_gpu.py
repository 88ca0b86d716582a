"""Calls of the gated delta memory that are allowed and easily overlooked."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, RESIDUAL, SOUP, SSC, make_delta_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from memory_caching_linear_gb300 import build
    build.build()
    mcl.load_library()


@pytest.mark.parametrize("mode", [GRM, SOUP, SSC])
@pytest.mark.parametrize("d,dtype", [(32, "f32"), (64, "bf16"), (128, "bf16")])
def test_one_segment_without_router_input(d, dtype, mode):
    L = 150
    q, k, v, _, la, be = (t.cuda() for t in make_delta_inputs(1, 2, L, d, L, d, dtype))
    dy = torch.randn_like(q)
    want, st = mcl.mc_forward_delta(q, k, v, None, la, be, L, RESIDUAL)
    for seg_len in (L, (1 << 32) + 5):  # a segment of more tokens than there are, past 32 bits too
        got, gst = mcl.mc_forward_delta(q, k, v, None, la, be, seg_len, mode, 2)
        assert torch.equal(got, want) and torch.equal(gst, st)
    grads = mcl.mc_backward_delta(q, k, v, None, la, be, dy, L, RESIDUAL)
    got = mcl.mc_backward_delta(q, k, v, None, la, be, dy, (1 << 32) + 5, mode, 2)
    assert not got[3].any()
    for g, w in zip(got[:3] + got[4:], grads[:3] + grads[4:]):
        assert torch.equal(g, w)
    leaf = [t.clone().requires_grad_() for t in (q, k, v, la, be)]
    mcl.DeltaMemoryCaching.apply(*leaf[:3], None, *leaf[3:], L, mode, 2).backward(dy)
    for t, w in zip(leaf, grads[:3] + grads[4:]):
        assert torch.equal(t.grad, w)


@pytest.mark.parametrize("C", [128, 70, 300])
def test_two_streams_at_once(C):
    """Calls on two streams share nothing: each has its own scratch."""
    xs = [[t.cuda() for t in make_delta_inputs(1, 4, 300 if C != 128 else 384, 64, C, s, "bf16")] for s in (1, 2)]
    dys = [torch.randn_like(x[0]) for x in xs]
    want = [mcl.mc_forward_delta(*x, C, GRM) for x in xs]
    grads = [mcl.mc_backward_delta(*x, dy, C, RESIDUAL) for x, dy in zip(xs, dys)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[i].append((mcl.mc_forward_delta(*xs[i], C, GRM), mcl.mc_backward_delta(*xs[i], dys[i], C, RESIDUAL)))
    torch.cuda.synchronize()
    for i in range(2):
        for fwd, bwd in out[i]:
            assert all(torch.equal(a, b) for a, b in zip(fwd, want[i]))
            assert all(a is b or torch.equal(a, b) for a, b in zip(bwd, grads[i]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_head_decodes_from_slices_of_its_sequence(dtype):
    """With B = H = 1 a token's slice is contiguous where it lies: log_alpha and beta at any element."""
    L, d, C = 9, 32, 4
    x = [t.cuda() for t in make_delta_inputs(1, 1, L, d, C, 17, dtype)]
    a, b = mcl.DecodeCache(1, 1, d, C, 4), mcl.DecodeCache(1, 1, d, C, 4)
    e, f = mcl.EvictingCache(1, 1, d, C, 2), mcl.EvictingCache(1, 1, d, C, 2)
    for j in range(L):
        tok = [t[:, :, j] for t in x]
        own = [t.clone() for t in tok]
        assert tok[4].is_contiguous() and (j == 0 or tok[4].data_ptr() != own[4].data_ptr())
        assert torch.equal(mcl.mc_decode_step_delta(a, *tok, GRM), mcl.mc_decode_step_delta(b, *own, GRM))
        got = mcl.mc_decode_step_evict(e, *tok[:4], GRM, log_alpha=tok[4], beta=tok[5])
        assert torch.equal(got, mcl.mc_decode_step_evict(f, *own[:4], GRM, log_alpha=own[4], beta=own[5]))


@pytest.mark.parametrize("C", [33, 11])
def test_parts_of_a_batch(C):
    """x[b:b + 1] of a batch is contiguous; its log_alpha and beta begin at any element."""
    x = [t.cuda() for t in make_delta_inputs(3, 1, 33, 64, C, 19, "bf16")]
    dy = torch.randn_like(x[0])
    y, st = mcl.mc_forward_delta(*x, C, GRM)
    grads = mcl.mc_backward_delta(*x, dy, C, RESIDUAL)
    for b in range(3):
        part = [t[b:b + 1] for t in x]
        assert b == 0 or part[4].data_ptr() % 16
        gy, gst = mcl.mc_forward_delta(*part, C, GRM)
        assert torch.equal(gy, y[b:b + 1]) and torch.equal(gst, st[b:b + 1])
        for g, w in zip(mcl.mc_backward_delta(*part, dy[b:b + 1], C, RESIDUAL), grads):
            assert w is None or torch.equal(g, w[b:b + 1])
        leaf = [t.clone().requires_grad_() for t in part[:3]]
        mcl.DeltaMemoryCaching.apply(*leaf, None, part[4], part[5], C, RESIDUAL, 0).backward(dy[b:b + 1])
        assert torch.equal(leaf[0].grad, grads[0][b:b + 1])
