"""The 64-bit forms that the gated delta memory's GPU tests compare against, checked on the CPU: against the
linear memory's oracle where the two rules meet, against closed forms, and their gradients against the
kernels' formulas and against differences."""
import numpy as np
import pytest
import torch

import oracle
from delta_ref import GRM, MEAN, RESIDUAL, SSC, Slots, backward, compact, forward, make_delta_inputs

MODES = [(RESIDUAL, 0), (GRM, 0), (SSC, 1), (MEAN, 0)]


@pytest.mark.parametrize("mode,topk", MODES)
def test_without_decay_or_error_it_is_the_linear_memory(mode, topk):
    # orthogonal keys within a segment: M k = 0 before the write, so e = v; beta = 1, no decay
    B, H, L, d, C = 1, 2, 40, 16, 16
    q, k, v, u, _, _ = make_delta_inputs(B, H, L, d, C, 1, "f32")
    eye = torch.eye(d).repeat(3, 1)[:L]
    k = eye.expand(B, H, L, d).contiguous()
    zero, one = torch.zeros(B, H, L), torch.ones(B, H, L)
    y, st = forward(q, k, v, u, zero, one, C, mode, topk)
    ref = oracle.forward(q, k, v, u, C, mode, topk)
    assert np.abs(y.numpy() - ref["y"]).max() < 1e-12
    assert np.abs(st.numpy() - ref["states"]).max() < 1e-12


def test_beta_one_and_unit_keys_store_the_value_exactly():
    q, k, v, u, la, _ = (x.double() for x in make_delta_inputs(1, 1, 12, 16, 12, 2, "f32"))
    k = k / k.norm(dim=-1, keepdim=True)
    y, st = forward(k, k, v, None, la, torch.ones_like(la), 12, RESIDUAL)  # read at the key just written
    assert (y - v).abs().max() < 1e-12


@pytest.mark.parametrize("mode,topk", MODES)
def test_gradients_against_differences(mode, topk):
    B, H, L, d, C = 1, 1, 14, 4, 5
    x = [t.double() for t in make_delta_inputs(B, H, L, d, C, 3, "f32")]
    dy = torch.randn(B, H, L, d, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    got = backward(*x, dy, C, mode, topk)
    h = 1e-6
    for n, (t, g) in enumerate(zip(x, got)):
        flat = t.reshape(-1)
        for i in range(0, flat.numel(), 7):
            keep = float(flat[i])
            f = []
            for step in (h, -h):
                flat[i] = keep + step
                f.append(float((forward(*x, C, mode, topk)[0] * dy).sum()))
            flat[i] = keep
            # central differences: h^2 / 6 of the third derivative and 1e-16 / h of rounding, both near 1e-9
            assert abs((f[0] - f[1]) / (2 * h) - float(g.reshape(-1)[i])) < 1e-6, (n, i)


def adjoint(q, k, v, la, be, p, R):
    """The kernels' formulas for one memory with the reads' gradients p [L, d] and the final state's R."""
    L, d = q.shape
    a = torch.exp(la)
    M, Ms, es = torch.zeros(d, d, dtype=torch.float64), [], []
    for t in range(L):
        M = a[t] * M
        e = v[t] - M @ k[t]
        M = M + be[t] * torch.outer(e, k[t])
        Ms.append(M)
        es.append(e)
    N = R.clone()
    h = float((R * Ms[-1]).sum())
    dq, dk, dv, dla, dbe = (torch.zeros_like(x) for x in (q, k, v, la, be))
    for t in range(L - 1, -1, -1):
        before = Ms[t - 1] if t else torch.zeros_like(M)
        dq[t] = Ms[t].T @ p[t]
        N = N + torch.outer(p[t], q[t])
        z = N @ k[t]
        w = be[t] * z
        dbe[t], dv[t] = z @ es[t], w
        dk[t] = be[t] * (N.T @ es[t]) - a[t] * (before.T @ w)
        N = a[t] * (N - torch.outer(w, k[t]))
        h = h + float(dq[t] @ q[t]) - float(w @ v[t])  # the decay's gradient as a running sum
        dla[t] = h
    return dq, dk, dv, dla, dbe


def test_gradients_against_the_formulas():
    L, d = 30, 8
    q, k, v, _, la, be = (x.double()[0, 0] for x in make_delta_inputs(1, 1, L, d, L, 5, "f32"))
    gen = torch.Generator().manual_seed(6)
    p, R = torch.randn(L, d, dtype=torch.float64, generator=gen), torch.randn(d, d, dtype=torch.float64, generator=gen)
    leaf = [x.clone().requires_grad_() for x in (q, k, v, la, be)]
    y, st = forward(*(x[None, None] for x in leaf[:3]), None, *(x[None, None] for x in leaf[3:]), L, RESIDUAL)
    want = torch.autograd.grad((y[0, 0] * p).sum() + (st[0, 0, 0] * R).sum(), leaf)
    for g, w in zip(adjoint(q, k, v, la, be, p, R), want):
        assert (g - w).abs().max() < 1e-11


def test_slots_that_never_fill_are_the_forward():
    B, H, L, d, C = 1, 2, 36, 8, 6
    x = make_delta_inputs(B, H, L, d, C, 7, "f32")
    y, st = forward(*x, C, SSC, 2)
    c = Slots(B, H, d, C, 6, 1)
    got = torch.stack([c.step(*(t[:, :, j] for t in x[:4]), SSC, 2, x[4][:, :, j], x[5][:, :, j]) for j in range(L)], 2)
    assert (got - y).abs().max() < 1e-12
    assert (c.states - st).abs().max() < 1e-12
    full, mass = compact(x[1], x[3], st, C, SSC, 2, 6, 1)
    assert torch.equal(full.slot_seg, c.slot_seg)
    assert (full.mass - c.mass).abs().max() < 1e-12 and (full.kbar - c.kbar).abs().max() < 1e-12
