"""Plain 64-bit forms of the gated delta memory, the evicting decode step and the compaction, token by
token, for the tests.  The forward is differentiable: autograd through it is one check of the gradients.

    e_t = v_t - a_t M_{t-1} k_t,  M_t = a_t M_{t-1} + beta_t e_t k_t^T,  a_t = exp(log_alpha_t)
"""
import math

import numpy as np
import torch

RESIDUAL, GRM, SOUP, SSC, MEAN = 0, 1, 2, 3, 4


def make_delta_inputs(B, H, L, d, C, seed, dtype, decay=0.05):
    """q, k, v, u [B, H, L, d], log_alpha, beta [B, H, L]: the keys of a segment share a direction and the
    router inputs lean towards one segment each, so that gates and masses are well apart."""
    rng = np.random.default_rng(seed)
    N = -(-L // C)
    topics = rng.standard_normal((B, H, N, d))
    topics /= np.linalg.norm(topics, axis=-1, keepdims=True)
    seg = np.arange(L) // C
    q = rng.standard_normal((B, H, L, d))
    q /= np.linalg.norm(q, axis=-1, keepdims=True)
    k = 0.7 * topics[:, :, seg] + rng.standard_normal((B, H, L, d)) / math.sqrt(d)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v = rng.standard_normal((B, H, L, d))
    want = rng.integers(0, N, (B, H, L, 1))
    u = 3 * np.take_along_axis(topics, want, 2) + rng.standard_normal((B, H, L, d)) / math.sqrt(d)
    la = -decay * np.exp(rng.standard_normal((B, H, L)))
    be = 1 / (1 + np.exp(-rng.standard_normal((B, H, L))))
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    return [torch.from_numpy(x).to(t).contiguous() for x in (q, k, v, u, la, be)]


def gates(k, u, C, mode, topk, given=None):
    """Gates [B, H, L, N] of the cached segments and [B, H, L] of the online one (64 bits)."""
    B, H, L, d = k.shape
    N = -(-L // C)
    kbar = [k[:, :, n * C:(n + 1) * C].mean(2) for n in range(N)]
    g, on = [], []
    for t in range(L):
        s = t // C
        if mode in (RESIDUAL, MEAN):
            w = 1.0 if mode == RESIDUAL else 1.0 / (s + 1)
            row = torch.zeros(B, H, N, dtype=k.dtype)
            row[..., :s] = w
            g.append(row)
            on.append(torch.full((B, H), w, dtype=k.dtype))
            continue
        r = [(u[:, :, t] * kbar[i]).sum(-1) for i in range(s)]
        r.append((u[:, :, t] * k[:, :, s * C:t + 1].mean(2)).sum(-1))
        r = torch.stack(r, -1)
        if mode == SSC and topk < min(s, N - 1):
            best = torch.sort(r[..., :s].detach(), dim=-1, descending=True, stable=True).indices[..., :topk]
            keep = torch.zeros(r.shape, dtype=torch.bool)
            keep.scatter_(-1, best, True)
            keep[..., s] = True
            r = r.masked_fill(~keep, -math.inf)
        w = torch.softmax(r, -1)
        g.append(torch.cat([w[..., :s], torch.zeros(B, H, N - s, dtype=k.dtype)], -1))
        on.append(w[..., s])
    return torch.stack(g, 2), torch.stack(on, 2)


def forward(q, k, v, u, la, be, C, mode, topk=0):
    """(y, states) in 64 bits."""
    q, k, v, la, be = (x.double() for x in (q, k, v, la, be))
    u = u.double() if u is not None else None
    B, H, L, d = q.shape
    N = -(-L // C)
    g, on = gates(k, u, C, mode, topk)
    a = torch.exp(la)
    cached, y = [], []
    for n in range(N):
        M = torch.zeros(B, H, d, d, dtype=torch.float64)
        for t in range(n * C, min(L, (n + 1) * C)):
            M = a[:, :, t, None, None] * M
            e = v[:, :, t] - (M @ k[:, :, t, :, None])[..., 0]
            M = M + (be[:, :, t, None] * e)[..., :, None] * k[:, :, t, None, :]
            read = on[:, :, t, None] * (M @ q[:, :, t, :, None])[..., 0]
            for i in range(n):
                read = read + g[:, :, t, i, None] * (cached[i] @ q[:, :, t, :, None])[..., 0]
            y.append(read)
        cached.append(M)
    return torch.stack(y, 2), torch.stack(cached, 2)


def backward(q, k, v, u, la, be, dy, C, mode, topk=0):
    """Gradients of <y, dy> by autograd through the token recurrence, in 64 bits: dq, dk, dv, du, dla, dbe."""
    leaf = [x.detach().double().clone().requires_grad_() if x is not None else None for x in (q, k, v, u, la, be)]
    y, _ = forward(*leaf, C, mode, topk)
    have = [x for x in leaf if x is not None]
    got = iter(torch.autograd.grad((y * dy.double()).sum(), have, allow_unused=True))
    out = []
    for x in leaf:
        if x is None:
            out.append(None)
            continue
        w = next(got)
        out.append(torch.zeros_like(x) if w is None else w)
    return out


class Slots:
    """The evicting cache of one (B, H) grid in 64 bits."""

    def __init__(self, B, H, d, C, n_max, protect):
        self.C, self.n_max, self.protect, self.t = C, n_max, protect, 0
        self.states = torch.zeros(B, H, n_max, d, d, dtype=torch.float64)
        self.kbar = torch.zeros(B, H, n_max, d, dtype=torch.float64)
        self.mass = torch.zeros(B, H, n_max, dtype=torch.float64)
        self.slot_seg = torch.full((B, H, n_max), -1, dtype=torch.int64)
        self.online = torch.zeros(B, H, d, d, dtype=torch.float64)
        self.ksum = torch.zeros(B, H, d, dtype=torch.float64)

    def step(self, q, k, v, u, mode, topk=0, la=None, be=None):
        q, k, v, u = (x.double() for x in (q, k, v, u))
        B, H, d = q.shape
        y = torch.zeros(B, H, d, dtype=torch.float64)
        s, pos = self.t // self.C, self.t % self.C
        for b in range(B):
            for h in range(H):
                if pos == 0:
                    self.online[b, h] = 0
                    self.ksum[b, h] = 0
                M = self.online[b, h]
                e = v[b, h]
                if la is not None:
                    M = M * math.exp(float(la[b, h]))
                    e = float(be[b, h]) * (e - M @ k[b, h])
                M = M + torch.outer(e, k[b, h])
                self.online[b, h] = M
                self.ksum[b, h] += k[b, h]
                held = [i for i in range(self.n_max) if self.slot_seg[b, h, i] >= 0]
                r = {i: float(self.kbar[b, h, i] @ u[b, h]) for i in held}
                if mode == SSC:
                    held = sorted(held, key=lambda i: (-r[i], int(self.slot_seg[b, h, i])))[:topk]
                on = float(self.ksum[b, h] @ u[b, h]) / (pos + 1)
                m = max([on] + [r[i] for i in held])
                z = math.exp(on - m) + sum(math.exp(r[i] - m) for i in held)
                y[b, h] = math.exp(on - m) / z * (M @ q[b, h])
                for i in held:
                    g = math.exp(r[i] - m) / z
                    y[b, h] += g * (self.states[b, h, i] @ q[b, h])
                    self.mass[b, h, i] += g
                if pos == self.C - 1:
                    ids = self.slot_seg[b, h].tolist()
                    empty = [i for i in range(self.n_max) if ids[i] < 0]
                    free = [i for i in range(self.n_max) if ids[i] < s - self.protect]
                    x = empty[0] if empty else min(free, key=lambda i: (float(self.mass[b, h, i]), ids[i]))
                    self.states[b, h, x], self.kbar[b, h, x] = M, self.ksum[b, h] / self.C
                    self.mass[b, h, x], self.slot_seg[b, h, x] = 0.0, s
        self.t += 1
        return y


def compact(k, u, states, C, mode, topk, n_max, protect):
    """The cache after a prefill, and every segment's mass."""
    B, H, L, d = k.shape
    k, u, states = k.double(), u.double(), states.double()
    N, done = -(-L // C), L // C
    g, _ = gates(k, u, C, mode, topk)
    mass = g.sum(2)
    c = Slots(B, H, d, C, n_max, protect)
    c.t = L
    for b in range(B):
        for h in range(H):
            new = list(range(max(0, done - protect), done))
            old = sorted(range(max(0, done - protect)), key=lambda i: (float(mass[b, h, i]), i))
            room = min(n_max, done) - len(new)
            kept = sorted(old[len(old) - room:] + new)
            for x, i in enumerate(kept):
                c.states[b, h, x], c.mass[b, h, x], c.slot_seg[b, h, x] = states[b, h, i], mass[b, h, i], i
                c.kbar[b, h, x] = k[b, h, i * C:(i + 1) * C].mean(0)
            if done < N:
                c.online[b, h] = states[b, h, N - 1]
                c.ksum[b, h] = k[b, h, done * C:].sum(0)
    return c, mass
