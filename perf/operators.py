"""Timing cases of the memory operators: the gated delta memory (forward over segments, its gradients, its
decoding step), decoding with a bounded cache that evicts by accumulated gate weight, and the compaction of a
prefill's segments into such a cache.

``run`` makes one pass, through the package where ``own`` is true and otherwise in plain torch operations; ``exact``
is the definition in 64 bits, token by token.  The memory, per (batch, head) and segment, from empty:

    e_t = v_t - a_t M_{t-1} k_t,   M_t = a_t M_{t-1} + beta_t e_t k_t^T,   a_t = exp(log_alpha_t)

and y_t = g_{t,s} M_t q_t + sum_{i<s} g_{t,i} M^(i) q_t with the gates of the aggregation: softmax of <u_t, mean key of
segment i> over the cached segments and the online one (keys up to t), or of the topk best cached ones (SSC).
"""
import torch

own = False

RESIDUAL, GRM, SSC = 0, 1, 3
CHUNK = 64  # tokens that the plain form takes at once


def listed():
    return [
        # one sequence of a small model, an odd length, the memory never cut: a plain gated delta layer in training
        dict(name="forward 1 head-group L1000", op="forward", B=1, H=4, L=1000, d=64, C=1000, mode=RESIDUAL, topk=0, dtype="bf16", states=False),
        # the long-context workload of the benchmark over the delta memory, as a prefill (the states are kept)
        dict(name="forward long grm", op="forward", B=1, H=16, L=65536, d=128, C=1024, mode=GRM, topk=0, dtype="bf16", states=True),
        # fp32 with a ragged last segment and the sparse router: an evaluation in full precision
        dict(name="forward f32 ssc ragged", op="forward", B=2, H=4, L=2000, d=64, C=250, mode=SSC, topk=2, dtype="f32", states=True),
        # a training step's gradients, the memory never cut: few long sequences
        dict(name="backward L4096 uncut", op="backward", B=2, H=16, L=4096, d=128, C=4096, mode=RESIDUAL, topk=0, dtype="bf16"),
        # a training step's gradients with cached segments and the router
        dict(name="backward grm L16384", op="backward", B=1, H=16, L=16384, d=128, C=1024, mode=GRM, topk=0, dtype="bf16"),
        # gradients in fp32, a ragged last segment, the sparse router
        dict(name="backward f32 ssc ragged", op="backward", B=1, H=4, L=1000, d=64, C=250, mode=SSC, topk=2, dtype="f32"),
        # one user's token stream on a small model: latency
        dict(name="decode one user", op="decode", B=1, H=4, d=64, C=256, n=5, mode=GRM, topk=0, dtype="bf16", tokens=8),
        # the benchmark's decoding shape: a batch over a nearly full cache
        dict(name="decode batch 63 cached", op="decode", B=8, H=16, d=128, C=256, n=63, mode=GRM, topk=0, dtype="bf16", tokens=8),
        # one user, a full cache, the step that completes a segment among the tokens
        dict(name="evict one user", op="evict", B=1, H=4, d=64, C=64, n=8, mode=SSC, topk=2, dtype="bf16", delta=False, tokens=8),
        # a batch over a full cache of delta memories; every head evicts its own segment
        dict(name="evict batch 32 slots", op="evict", B=8, H=16, d=128, C=256, n=32, mode=GRM, topk=0, dtype="bf16", delta=True, tokens=8),
        # a short prompt in fp32 into a few slots
        dict(name="compact f32 short", op="compact", B=2, H=8, L=4000, d=64, C=256, keep=6, protect=1, mode=GRM, topk=0, dtype="f32"),
        # a long prompt of 128 segments into a cache of 32
        dict(name="compact long", op="compact", B=1, H=16, L=65536, d=128, C=512, keep=32, protect=2, mode=GRM, topk=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["forward", "backward", "decode", "evict", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 32] if dtype == "bf16" else [16, 32, 64, 128])
    mode = rng.choice([GRM, GRM, SSC])
    if op in ("forward", "backward"):
        top = (1 << 27) if op == "forward" else (1 << 24)  # values of one tensor [B, H, L, d]
        if dtype == "f32":
            top >>= 6
        L = _log_int(rng, 33, 16384 if dtype == "bf16" else 3000)
        bh = max(1, min(64, top // (L * d)))
        H = rng.randint(1, max(1, min(16, bh)))
        B = rng.randint(1, max(1, min(4, bh // H)))
        kind = rng.choice(["uncut", "tiles", "odd"])
        if kind == "uncut":
            C, mode = L, RESIDUAL
        elif kind == "tiles":
            C = 128 * _log_int(rng, 1, 16)
        else:
            C = _log_int(rng, 17, 1500)
        if mode == SSC:
            L = min(L, 4096)
        C = max(C, -(-L // 48))
        mode = RESIDUAL if C >= L else rng.choice([mode, mode, mode, RESIDUAL])  # a single memory has nothing to weigh
        case = dict(op=op, B=B, H=H, L=L, d=d, C=min(C, L), mode=mode, topk=rng.randint(1, 6) if mode == SSC else 0, dtype=dtype)
        if op == "forward":
            case["states"] = rng.random() < 0.5
        return case
    if op in ("decode", "evict"):
        n = rng.randint(2, 63)
        C = _log_int(rng, 16, 1024)
        case = dict(op=op, B=rng.randint(1, 8), H=rng.randint(1, 16), d=d, C=C, n=n if op == "decode" else min(n, 32),
                    mode=mode, topk=rng.randint(1, 6) if mode == SSC else 0, dtype=dtype, tokens=rng.randint(2, 8))
        if op == "evict":
            case["delta"] = rng.random() < 0.5
        return case
    C = _log_int(rng, 16, 1024)
    n = rng.randint(3, 120)
    L = min(65536, C * n + rng.randint(0, C - 1))
    H = rng.randint(1, 16)
    n = L // C
    keep = rng.randint(2, max(2, min(n, 64)))
    return dict(op="compact", B=1, H=H, L=L, d=d, C=C, keep=keep, protect=rng.randint(0, min(2, keep)), mode=GRM, topk=0, dtype=dtype)


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _sequence(case, g):
    """q, k, v, u [B, H, L, d] as a trained router meets them: the keys of a segment share a topic, and each token asks
    for one topic, some far more often than others."""
    B, H, L, d, C = (case[x] for x in ("B", "H", "L", "d", "C"))
    dev, t = "cuda", _dtype(case)
    N = -(-L // C)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    q, v = _unit(rnd(B, H, L, d)), rnd(B, H, L, d)
    topics = _unit(rnd(B, H, N, d))
    seg = torch.arange(L, device=dev) // C
    k = _unit(topics[:, :, seg] * 0.7 + rnd(B, H, L, d) * (d ** -0.5))
    liked = torch.multinomial(torch.softmax(rnd(B * H, N), -1), L, replacement=True, generator=g).view(B, H, L, 1)
    u = 3.0 * torch.gather(topics, 2, liked.expand(B, H, L, d)) + rnd(B, H, L, d) * (d ** -0.5)
    return [x.to(t).contiguous() for x in (q, k, v, u)]


def _gates(case, shape, g):
    t = _dtype(case)
    log_alpha = -0.02 * torch.exp(torch.randn(*shape, device="cuda", generator=g))
    beta = torch.sigmoid(torch.randn(*shape, device="cuda", generator=g))
    return log_alpha.to(t).contiguous(), beta.to(t).contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op in ("forward", "backward"):
        s["q"], s["k"], s["v"], s["u"] = _sequence(case, g)
        if case["mode"] == RESIDUAL:
            s["u"] = None  # no router
        s["log_alpha"], s["beta"] = _gates(case, (case["B"], case["H"], case["L"]), g)
        if op == "backward":
            s["dy"] = torch.randn(s["q"].shape, device="cuda", generator=g).to(s["q"].dtype)
        return s
    if op == "compact":
        s["k"], s["u"] = _sequence(case, g)[1::2]
        N = -(-case["L"] // case["C"])
        s["states"] = torch.randn(case["B"], case["H"], N, case["d"], case["d"], device="cuda", generator=g)
        if own:
            import memory_caching_linear_gb300 as mcl
            s["cache"] = mcl.EvictingCache(case["B"], case["H"], case["d"], case["C"], case["keep"], protect=case["protect"])
        return s
    # a decoding cache of n completed segments: "decode" begins a segment, "evict" goes over a segment's end
    B, H, d, C, n, T = (case[x] for x in ("B", "H", "d", "C", "n", "tokens"))
    rnd = lambda *x: torch.randn(*x, device="cuda", generator=g)  # noqa: E731
    t = _dtype(case)
    s["states"] = rnd(B, H, n, d, d) * 0.5
    s["kbar"] = _unit(rnd(B, H, n, d)) * 0.6
    s["online"] = rnd(B, H, d, d) * 0.3
    toks = []
    for _ in range(T):
        q, k, v = _unit(rnd(B, H, d)), _unit(rnd(B, H, d)), rnd(B, H, d)
        liked = torch.randint(0, n, (B, H, 1, 1), device="cuda", generator=g)
        u = 5.0 * torch.gather(s["kbar"], 2, liked.expand(B, H, 1, d))[:, :, 0] + rnd(B, H, d) * (d ** -0.5)
        la, be = _gates(case, (B, H), g)
        toks.append([x.to(t).contiguous() for x in (q, k, v, u)] + [la, be])
    s["toks"] = toks
    if op == "decode":
        s["t0"] = n * C
        s["ksum"] = torch.zeros(B, H, d, device="cuda")
    else:
        done = n + 7  # segments completed so far: seven are gone already
        s["t0"] = done * C + max(0, C - max(1, T // 2))
        s["ksum"] = rnd(B, H, d) * 0.5 + (s["t0"] % C) * 0.05
        order = torch.argsort(torch.rand(B, H, done - 1, device="cuda", generator=g), -1)[..., :n - 1]
        last = torch.full((B, H, 1), done - 1, device="cuda", dtype=order.dtype)
        s["slot_seg"] = torch.cat([order, last], -1).to(torch.int32).contiguous()  # slots in no order; the newest is there
        s["mass"] = torch.rand(B, H, n, device="cuda", generator=g) * 40.0
    if own:
        import memory_caching_linear_gb300 as mcl
        if op == "decode":
            c = mcl.DecodeCache(B, H, d, C, n + 1)
            c.states[:, :, :n], c.kbar[:, :, :n] = s["states"], s["kbar"]
            s["cache"] = c
        else:
            c = mcl.EvictingCache(B, H, d, C, n, protect=1)
            for name in ("states", "kbar", "online", "ksum", "mass", "slot_seg"):
                getattr(c, name).copy_(s[name])
            c.t = s["t0"]
            s["prompt"] = c  # the cache after the prompt, from which each continuation starts
            s["cache"] = mcl.EvictingCache(B, H, d, C, n, protect=1)
    return s


# ----------------------------------------------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------------------------------------------
def _split(x, C, fill=0.0):
    """[B, H, L, ...] -> [B*H, N, chunks, CHUNK, ...] in fp32: segments of C tokens, each filled up to whole chunks."""
    B, H, L = x.shape[:3]
    N, Cp = -(-L // C), -(-C // CHUNK) * CHUNK
    x = x.reshape(B * H, L, *x.shape[3:]).float()
    pad = torch.full((B * H, N * C - L, *x.shape[2:]), fill, device=x.device)
    x = torch.cat([x, pad], 1).reshape(B * H, N, C, *x.shape[2:])
    pad = torch.full((B * H, N, Cp - C, *x.shape[3:]), fill, device=x.device)
    return torch.cat([x, pad], 2).reshape(B * H, N, Cp // CHUNK, CHUNK, *x.shape[3:])


def _join(x, C, L):
    """The inverse of _split: [BH, N, chunks, CHUNK, ...] -> [BH, L, ...]."""
    BH, N = x.shape[:2]
    x = x.reshape(BH, N, -1, *x.shape[4:])[:, :, :C]
    return x.reshape(BH, N * C, *x.shape[3:])[:, :L]


def _delta_chunks(q, k, v, log_alpha, beta, C):
    """The delta memory in chunks: online reads [BH, L, d] and every segment's final state [BH, N, d, d]."""
    L = q.shape[2]
    Q, K, V, A, Bt = (_split(x, C) for x in (q, k, v, log_alpha, beta))
    cum = A.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]) * low) * low
    eye = torch.eye(CHUNK, device=q.device, dtype=torch.float64)
    X = -(K @ K.transpose(-1, -2)).double() * (decay * Bt[..., None, :]) * (1 - eye)
    T = eye + X  # in 64 bits: the powers of keys that resemble each other grow before they vanish
    for _ in range(5):  # (I - X)^-1 = (I + X)(I + X^2)(I + X^4)...: X^64 = 0
        X = X @ X
        T = T + T @ X
    T = T.float()
    P = (Q @ K.transpose(-1, -2)) * decay
    gam = torch.exp(cum)[..., None]
    last = cum[..., -1:]
    tail = (torch.exp(last - cum) * Bt)[..., None]
    S = torch.zeros(*Q.shape[:2], Q.shape[-1], Q.shape[-1], device=q.device)
    outs = []
    for c in range(Q.shape[2]):
        St = S.transpose(-1, -2)
        E = T[:, :, c] @ (V[:, :, c] - gam[:, :, c] * (K[:, :, c] @ St))
        outs.append(gam[:, :, c] * (Q[:, :, c] @ St) + P[:, :, c] @ (Bt[:, :, c, :, None] * E))
        S = torch.exp(last[:, :, c])[..., None] * S + (tail[:, :, c] * E).transpose(-1, -2) @ K[:, :, c]
    return _join(torch.stack(outs, 2), C, L), S


def _scores(k, u, C):
    """Router scores in 64 bits (near-equal ones are ranked): cached [BH, L, N] and online [BH, L]."""
    B, H, L, d = k.shape
    N = -(-L // C)
    kd, ud = k.reshape(B * H, L, d).double(), u.reshape(B * H, L, d).double()
    seg = torch.arange(L, device=k.device) // C
    run = kd.cumsum(1)
    ends = torch.clamp((torch.arange(N, device=k.device) + 1) * C, max=L) - 1
    at_end = run[:, ends]
    before = torch.cat([torch.zeros_like(at_end[:, :1]), at_end[:, :-1]], 1)
    size = (ends + 1 - torch.arange(N, device=k.device) * C).double()
    kbar = (at_end - before) / size[:, None]
    count = (torch.arange(L, device=k.device) % C + 1).double()
    pooled = (run - before[:, seg]) / count[:, None]
    return ud @ kbar.transpose(-1, -2), (ud * pooled).sum(-1), seg, kbar


def _weights(r, r_on, seg, mode, topk):
    """Gates: cached [BH, L, N] (zero where a segment is not read) and online [BH, L]."""
    N = r.shape[-1]
    cached = torch.arange(N, device=r.device)[None] < seg[:, None]
    r = r.masked_fill(~cached, float("-inf"))
    if mode == SSC and topk < N - 1:
        rank = torch.argsort(torch.argsort(r.detach(), dim=-1, descending=True, stable=True), -1)
        r = r.masked_fill(rank >= topk, float("-inf"))
    z = torch.cat([r, r_on[..., None]], -1)
    w = torch.exp(z - z.detach().amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    return w[..., :N], w[..., N]


def _plain_forward(q, k, v, u, log_alpha, beta, case):
    B, H, L, d = q.shape
    C, mode = case["C"], case["mode"]
    y, S = _delta_chunks(q, k, v, log_alpha, beta, C)
    N = S.shape[1]
    if mode == RESIDUAL:
        w, w_on = None, None
    else:
        w, w_on = (x.float() for x in _weights(*_scores(k, u, C)[:3], mode, case["topk"]))
        y = w_on[..., None] * y
    qf = q.reshape(B * H, L, d).float()
    for i in range(N - 1):  # one cached memory at a time, read by every later token
        t = (i + 1) * C
        read = qf[:, t:] @ S[:, i].transpose(-1, -2)
        y = torch.cat([y[:, :t], y[:, t:] + (read if w is None else w[:, t:, i, None] * read)], 1)
    return y.reshape(B, H, L, d).to(q.dtype), S.reshape(B, H, N, d, d)


def _plain_decode(s):
    """tokens steps from the prepared cache; nothing of it is written."""
    B, H, d, C, n, mode, topk = (s[x] for x in ("B", "H", "d", "C", "n", "mode", "topk"))
    evict = s["op"] == "evict"
    delta = not evict or s["delta"]
    states, kbar, online, ksum = s["states"], s["kbar"], s["online"], s["ksum"]
    slot_seg, mass = (s["slot_seg"], s["mass"]) if evict else (None, None)
    ys = []
    for j, (q, k, v, u, la, be) in enumerate(s["toks"]):
        t = s["t0"] + j
        seg, pos = t // C, t % C
        qf, kf, vf, uf = (x.float() for x in (q, k, v, u))
        if pos == 0:
            online, ksum = torch.zeros_like(online), torch.zeros_like(ksum)
        if delta:
            M = torch.exp(la.float())[..., None, None] * online
            e = be.float()[..., None] * (vf - (M @ kf[..., None])[..., 0])
        else:
            M, e = online, vf
        online = M + e[..., None] * kf[..., None, :]
        ksum = ksum + kf
        r = (kbar.double() @ uf.double()[..., None])[..., 0]
        r_on = (uf.double() * ksum.double()).sum(-1) / (pos + 1)
        if mode == SSC and topk < n:
            # the best scores; equal ones to the older segment
            by = torch.argsort(slot_seg, -1) if evict else torch.arange(n, device=r.device).expand(B, H, n)
            rank = torch.argsort(torch.argsort(torch.gather(r, -1, by), dim=-1, descending=True, stable=True), -1)
            rank = torch.zeros_like(rank).scatter(-1, by, rank)
            r = r.masked_fill(rank >= topk, float("-inf"))
        z = torch.cat([r, r_on[..., None]], -1)
        w = torch.exp(z - z.amax(-1, keepdim=True))
        w = (w / w.sum(-1, keepdim=True)).float()
        read = (states.reshape(B, H, n * d, d) @ qf[..., None]).reshape(B, H, n, d)
        ys.append((w[..., n, None] * (online @ qf[..., None])[..., 0] + (w[..., :n, None] * read).sum(-2)).to(q.dtype))
        if evict:
            mass = mass + w[..., :n]
            if pos == C - 1:  # the new segment takes the slot of the one with the least weight, the newest spared
                free = slot_seg < seg - 1
                out = mass.masked_fill(~free, float("inf"))
                low = out.amin(-1, keepdim=True)
                out = torch.where(out == low, slot_seg, 1 << 30).argmin(-1)
                hit = torch.arange(n, device=r.device) == out[..., None]
                states = torch.where(hit[..., None, None], online[:, :, None], states)
                kbar = torch.where(hit[..., None], (ksum / C)[:, :, None], kbar)
                mass = mass.masked_fill(hit, 0.0)
                slot_seg = torch.where(hit, seg, slot_seg).to(torch.int32)
    got = {"y": ys, "online": online, "ksum": ksum}
    if evict:
        got |= {"states": states, "kbar": kbar, "mass": mass, "slot_seg": slot_seg}
    return got


def _plain_compact(s, k, u, states):
    B, H, L, d = k.shape
    C, keep, protect = s["C"], s["keep"], s["protect"]
    done = L // C
    r, r_on, seg, kbar = _scores(k, u, C)
    w, _ = _weights(r, r_on, seg, s["mode"], s["topk"])
    mass = w.sum(1)  # [BH, N] in 64 bits
    rank = mass[:, :done].clone()
    rank[:, done - protect:done] = float("inf")
    # the least go first, equal ones the older first
    gone = torch.argsort(torch.argsort(rank, dim=-1, stable=True), -1) < done - keep
    kept = torch.argsort(gone.to(torch.int8), dim=-1, stable=True)[:, :keep]
    rows = torch.arange(B * H, device=k.device)[:, None]
    flat = states.reshape(B * H, -1, d, d)
    part = L % C > 0
    online = flat[:, -1] if part else torch.zeros_like(flat[:, 0])
    ksum = k.reshape(B * H, L, d)[:, done * C:].double().sum(1)
    return {"states": flat[rows, kept].reshape(B, H, keep, d, d), "kbar": kbar[rows, kept].float().reshape(B, H, keep, d),
            "mass": mass[rows, kept].float().reshape(B, H, keep), "slot_seg": kept.to(torch.int32).reshape(B, H, keep),
            "online": online.reshape(B, H, d, d).clone(), "ksum": ksum.float().reshape(B, H, d),
            "all": mass.float().reshape(B, H, -1)}


def run(s):
    op = s["op"]
    if own:
        import memory_caching_linear_gb300 as mcl
        if op == "forward":
            y, states = mcl.mc_forward_delta(s["q"], s["k"], s["v"], s["u"], s["log_alpha"], s["beta"], s["C"], s["mode"],
                                             s["topk"], want_states=s["states"])
            return (y, states) if s["states"] else y
        if op == "backward":
            got = mcl.mc_backward_delta(s["q"], s["k"], s["v"], s["u"], s["log_alpha"], s["beta"], s["dy"], s["C"],
                                        s["mode"], s["topk"])
            return {n: x for n, x in zip(("dq", "dk", "dv", "du", "dlog_alpha", "dbeta"), got) if x is not None}
        c = s["cache"]
        if op == "compact":
            mass = mcl.mc_cache_compact(c, s["k"], s["u"], s["states"], s["mode"], s["topk"])
            return {"states": c.states, "kbar": c.kbar, "mass": c.mass, "slot_seg": c.slot_seg, "online": c.online,
                    "ksum": c.ksum, "all": mass}
        if op == "decode":
            c.t = s["t0"]
            ys = [mcl.mc_decode_step_delta(c, q, k, v, u, la, be, s["mode"], s["topk"]) for q, k, v, u, la, be in s["toks"]]
            return {"y": ys, "online": c.online, "ksum": c.ksum}
        c.copy_(s["prompt"])
        ys = [mcl.mc_decode_step_evict(c, q, k, v, u, s["mode"], s["topk"], log_alpha=la if s["delta"] else None,
                                       beta=be if s["delta"] else None) for q, k, v, u, la, be in s["toks"]]
        return {"y": ys, "online": c.online, "ksum": c.ksum, "states": c.states, "kbar": c.kbar, "mass": c.mass,
                "slot_seg": c.slot_seg}
    if op == "forward":
        y, states = _plain_forward(s["q"], s["k"], s["v"], s["u"], s["log_alpha"], s["beta"], s)
        return (y, states) if s["states"] else y
    if op == "backward":
        names = ["q", "k", "v", "u", "log_alpha", "beta"]
        if s["u"] is None:
            names.remove("u")
        leaf = {n: s[n].detach().float().requires_grad_() for n in names}
        y, _ = _plain_forward(leaf["q"], leaf["k"], leaf["v"], leaf.get("u"), leaf["log_alpha"], leaf["beta"], s)
        got = torch.autograd.grad(y, [leaf[n] for n in names], s["dy"].float())
        return {"d" + n: x.to(s["q"].dtype) for n, x in zip(names, got)}
    if op == "compact":
        return _plain_compact(s, s["k"], s["u"], s["states"])
    return _plain_decode(s)


# ----------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    B, H, d, C = case["B"], case["H"], case["d"], case["C"]
    BH = B * H
    if op in ("forward", "backward"):
        L, routed = case["L"], case["mode"] != RESIDUAL
        N = -(-L // C)
        seg_reads = sum((min(L, (s + 1) * C) - s * C) * (min(s, case["topk"]) if case["mode"] == SSC else s) for s in range(N))
        if not routed:
            seg_reads = L if N > 1 else 0  # constant gates: the cached memories add up to one
        # per token: the read of M k, its rank-one update, the read of M q; cached reads; scores
        flops = BH * (6 * d * d * L + 2 * d * d * seg_reads + (2 * d * sum(min(L, (s + 1) * C) - s * C for s in range(N)) * (N + 1) // 2 if routed else 0))
        tensors = 4 + (1 if routed else 0)
        if op == "forward":
            return {"bytes": BH * (tensors * L * d * e + 2 * L * e + (4 * N * d * d if case["states"] else 0)), "flops": flops}
        return {"bytes": BH * ((2 * tensors - 1) * L * d * e + 4 * L * e), "flops": 3 * flops}
    if op == "compact":
        L, keep = case["L"], case["keep"]
        N = -(-L // C)
        reads = sum((min(L, (s + 1) * C) - s * C) * (s + 1) for s in range(N))
        return {"bytes": BH * (2 * L * d * e + 2 * (keep + (1 if L % C else 0)) * 4 * d * d + 4 * keep * d), "flops": BH * 2 * d * reads}
    n, T = case["n"], case["tokens"]
    # each token reads every memory that its gates weigh and updates the online one
    read = min(n, case["topk"]) if case["mode"] == SSC else n
    state = 4 * d * d
    moved = T * (read * state + 2 * state + 4 * n * d + 5 * d * e)
    if op == "evict":
        moved += 2 * n * state + state  # each continuation starts from a copy of the prompt's cache
    return {"bytes": BH * moved, "flops": BH * T * 2 * d * d * (read + 4)}


# ----------------------------------------------------------------------------------------------------------------
# the definition, token by token, in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def _by_segment(x, C, fill=0.0):
    """[B, H, L, ...] -> [B*H*N, C, ...] in 64 bits, the last segment filled with tokens that change nothing."""
    B, H, L = x.shape[:3]
    N = -(-L // C)
    out = torch.full((B * H, N * C, *x.shape[3:]), fill, device=x.device, dtype=torch.float64)
    out[:, :L] = x.reshape(B * H, L, *x.shape[3:]).double()
    return out.reshape(B * H * N, C, *x.shape[3:])


def _recur(s, keep):
    """All segments side by side, one token at a time: errors e [R, C, d], reads [R, C, d], final states, and (keep) M_t."""
    C = s["C"]
    q, k, v = (_by_segment(s[n], C) for n in "qkv")
    a, b = torch.exp(_by_segment(s["log_alpha"], C)), _by_segment(s["beta"], C)
    R, d = q.shape[0], q.shape[-1]
    M = torch.zeros(R, d, d, device=q.device, dtype=torch.float64)
    every = torch.empty(C, R, d, d, device=q.device, dtype=torch.float64) if keep else None
    err, out = torch.empty_like(v), torch.empty_like(v)
    for t in range(C):
        M *= a[:, t, None, None]
        e = v[:, t] - torch.bmm(M, k[:, t, :, None])[..., 0]
        M.baddbmm_((b[:, t, None] * e)[:, :, None], k[:, t, None, :])
        out[:, t] = torch.bmm(M, q[:, t, :, None])[..., 0]
        err[:, t] = e
        if keep:
            every[t] = M
    return q, k, v, a, b, err, out, M, every


def _gates64(k, u, C, mode, topk):
    """Per (batch, head): gates of the cached segments, online gate, pooled keys of each token, key means."""
    B, H, L, d = k.shape
    N, dev = -(-L // C), k.device
    kk, uu = k.reshape(B * H, L, d).double(), u.reshape(B * H, L, d).double()
    pool, mean = torch.empty_like(kk), torch.empty(B * H, N, d, device=dev, dtype=torch.float64)
    for n in range(N):
        part = kk[:, n * C:(n + 1) * C]
        pool[:, n * C:(n + 1) * C] = part.cumsum(1) / torch.arange(1, part.shape[1] + 1, device=dev)[:, None]
        mean[:, n] = part.mean(1)
    g, g_on = torch.zeros(B * H, L, N, device=dev, dtype=torch.float64), torch.empty(B * H, L, device=dev, dtype=torch.float64)
    for n in range(N):
        x = uu[:, n * C:(n + 1) * C]
        on = (x * pool[:, n * C:(n + 1) * C]).sum(-1, keepdim=True)
        r = x @ mean[:, :n].transpose(1, 2)
        if mode == SSC and topk < min(n, N - 1):
            best = torch.sort(r, dim=-1, descending=True, stable=True).indices[..., :topk]
            r = torch.full_like(r, float("-inf")).scatter(-1, best, torch.gather(r, -1, best))
        w = torch.softmax(torch.cat([r, on], -1), -1)
        g[:, n * C:(n + 1) * C, :n], g_on[:, n * C:(n + 1) * C] = w[..., :-1], w[..., -1]
    return g, g_on, pool, mean


def _exact_forward(s):
    B, H, L, d, C = (s[x] for x in ("B", "H", "L", "d", "C"))
    N = -(-L // C)
    out, M = _recur(s, False)[6:8]
    y, S = out.reshape(B * H, N * C, d)[:, :L].clone(), M.reshape(B * H, N, d, d)
    if s["mode"] != RESIDUAL:
        g, g_on = _gates64(s["k"], s["u"], C, s["mode"], s["topk"])[:2]
        y *= g_on[..., None]
    q = s["q"].reshape(B * H, L, d).double()
    if s["mode"] == RESIDUAL:
        acc = S.cumsum(1)
        for n in range(1, N):
            y[:, n * C:(n + 1) * C] += q[:, n * C:(n + 1) * C] @ acc[:, n - 1].transpose(1, 2)
    else:
        for n in range(1, N):
            for i in range(n):
                y[:, n * C:(n + 1) * C] += g[:, n * C:(n + 1) * C, i, None] * (q[:, n * C:(n + 1) * C] @ S[:, i].transpose(1, 2))
    y = y.reshape(B, H, L, d)
    return (y, S.reshape(B, H, N, d, d)) if s["states"] else y


def _exact_backward(s):
    B, H, L, d, C = (s[x] for x in ("B", "H", "L", "d", "C"))
    N, routed = -(-L // C), s["mode"] != RESIDUAL
    if B * H * N * C * d * d * 8 > 6e10:
        return None
    q, k, v, a, b, err, out, M, every = _recur(s, True)
    dy = _by_segment(s["dy"], C)
    BH, S = B * H, M.reshape(B * H, N, d, d)
    flat = lambda x: x.reshape(BH, N * C, *x.shape[2:])[:, :L]  # noqa: E731
    qf, dyf = flat(q), flat(dy)
    dq, du = torch.zeros(BH, L, d, device=q.device, dtype=torch.float64), None
    G = torch.zeros_like(S)
    dk_pool = torch.zeros(BH, N * C, d, device=q.device, dtype=torch.float64)
    g_on = torch.ones(BH, L, device=q.device, dtype=torch.float64)
    if routed:
        u = s["u"].reshape(BH, L, d).double()
        g, g_on, pool, mean = _gates64(s["k"], s["u"], C, s["mode"], s["topk"])
        dg = torch.zeros_like(g)
    for i in range(N - 1):
        t = (i + 1) * C
        w = g[:, t:, i, None] if routed else 1.0
        if routed:
            dg[:, t:, i] = (dyf[:, t:] * (qf[:, t:] @ S[:, i].transpose(1, 2))).sum(-1)
        dq[:, t:] += w * (dyf[:, t:] @ S[:, i])
        G[:, i] = (w * dyf[:, t:]).transpose(1, 2) @ qf[:, t:]
    if routed:
        dg_on = (dyf * flat(out)).sum(-1)
        mid = (g * dg).sum(-1) + g_on * dg_on
        dr, dr_on = g * (dg - mid[..., None]), g_on * (dg_on - mid)
        du = dr @ mean + dr_on[..., None] * pool
        dmean = dr.transpose(1, 2) @ u
        for n in range(N):
            lo, hi = n * C, min(L, (n + 1) * C)
            share = (dr_on[:, lo:hi] / torch.arange(1, hi - lo + 1, device=q.device))[..., None] * u[:, lo:hi]
            dk_pool[:, lo:hi] = share.flip(1).cumsum(1).flip(1) + dmean[:, n, None] / (hi - lo)
    gs = torch.ones(BH, N * C, device=q.device, dtype=torch.float64)
    gs[:, :L] = g_on
    do = dy * gs.reshape(BH * N, C, 1)
    W = G.reshape(BH * N, d, d).clone()  # the adjoint of M_t, walked back
    dqs, dks, dvs = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    da, db = torch.empty_like(a), torch.empty_like(b)
    zero = torch.zeros_like(W)
    for t in range(C - 1, -1, -1):
        before = every[t - 1] if t else zero
        dqs[:, t] = torch.bmm(every[t].transpose(1, 2), do[:, t, :, None])[..., 0]
        W.baddbmm_(do[:, t, :, None], q[:, t, None, :])
        z = torch.bmm(W, k[:, t, :, None])[..., 0]
        db[:, t] = (z * err[:, t]).sum(-1)
        w = b[:, t, None] * z
        dvs[:, t] = w
        dks[:, t] = (torch.bmm(W.transpose(1, 2), (b[:, t, None] * err[:, t])[..., None])
                     - a[:, t, None, None] * torch.bmm(before.transpose(1, 2), w[..., None]))[..., 0]
        W.baddbmm_(w[:, :, None], k[:, t, None, :], alpha=-1)
        W *= a[:, t, None, None]
        da[:, t] = (W * before).sum((1, 2))  # the gradient of log alpha
    shape = (B, H, L, d)
    got = {"dq": (flat(dqs) + dq).reshape(shape), "dk": (flat(dks) + dk_pool[:, :L]).reshape(shape), "dv": flat(dvs).reshape(shape)}
    if routed:
        got["du"] = du.reshape(shape)
    return got | {"dlog_alpha": flat(da).reshape(B, H, L), "dbeta": flat(db).reshape(B, H, L)}


def _exact_decode(s):
    B, H, d, C, n, mode, topk = (s[x] for x in ("B", "H", "d", "C", "n", "mode", "topk"))
    evict = s["op"] == "evict"
    R = B * H
    M, mean = s["states"].double().reshape(R, n, d, d).clone(), s["kbar"].double().reshape(R, n, d).clone()
    on, total = s["online"].double().reshape(R, d, d).clone(), s["ksum"].double().reshape(R, d).clone()
    ids = s["slot_seg"].reshape(R, n).long().clone() if evict else torch.arange(n, device=M.device).expand(R, n)
    mass = s["mass"].double().reshape(R, n).clone() if evict else None
    ys = []
    for j, tok in enumerate(s["toks"]):
        t = s["t0"] + j
        q, k, v, u = (x.double().reshape(R, d) for x in tok[:4])
        if t % C == 0:
            on.zero_()
            total.zero_()
        if not evict or s["delta"]:
            on *= torch.exp(tok[4].double()).reshape(R, 1, 1)
            v = tok[5].double().reshape(R, 1) * (v - torch.einsum("rij,rj->ri", on, k))
        on += torch.einsum("ri,rj->rij", v, k)
        total += k
        r = torch.einsum("rnj,rj->rn", mean, u)
        if mode == SSC and topk < n:
            first = torch.argsort(ids, -1)
            best = torch.sort(torch.gather(r, 1, first), dim=-1, descending=True, stable=True).indices[:, :topk]
            best = torch.gather(first, 1, best)
            r = torch.full_like(r, float("-inf")).scatter(1, best, torch.gather(r, 1, best))
        w = torch.softmax(torch.cat([r, (u * total).sum(-1, keepdim=True) / (t % C + 1)], -1), -1)
        y = torch.einsum("rn,rnij,rj->ri", w[:, :n], M, q) + w[:, n, None] * torch.einsum("rij,rj->ri", on, q)
        ys.append(y.reshape(B, H, d))
        if evict:
            mass += w[:, :n]
            if t % C == C - 1:
                for h in range(R):
                    allowed = [x for x in range(n) if int(ids[h, x]) < t // C - 1]
                    x = min(allowed, key=lambda x: (float(mass[h, x]), int(ids[h, x])))
                    M[h, x], mean[h, x], mass[h, x], ids[h, x] = on[h], total[h] / C, 0.0, t // C
    got = {"y": ys, "online": on.reshape(B, H, d, d), "ksum": total.reshape(B, H, d)}
    if evict:
        got |= {"states": M.reshape(B, H, n, d, d), "kbar": mean.reshape(B, H, n, d), "mass": mass.reshape(B, H, n),
                "slot_seg": ids.reshape(B, H, n).to(torch.int32)}
    return got


def _exact_compact(s):
    B, H, L, d = s["k"].shape
    C, keep, protect = s["C"], s["keep"], s["protect"]
    done, N = L // C, -(-L // C)
    g, _, _, mean = _gates64(s["k"], s["u"], C, s["mode"], s["topk"])
    mass = g.sum(1)
    slots = []
    for row in mass.tolist():
        loose = sorted(range(done - protect), key=lambda i: (row[i], i))
        slots.append(sorted(loose[done - keep:] + list(range(done - protect, done))))
    slots = torch.tensor(slots, device=mass.device)
    rows = torch.arange(B * H, device=mass.device)[:, None]
    states = s["states"].reshape(B * H, N, d, d).double()
    online = states[:, -1] if L % C else torch.zeros_like(states[:, 0])
    tail = s["k"].reshape(B * H, L, d)[:, done * C:].double().sum(1)
    return {"states": states[rows, slots].reshape(B, H, keep, d, d), "kbar": mean[rows, slots].reshape(B, H, keep, d),
            "mass": mass[rows, slots].reshape(B, H, keep), "slot_seg": slots.to(torch.int32).reshape(B, H, keep),
            "online": online.reshape(B, H, d, d), "ksum": tail.reshape(B, H, d), "all": mass.reshape(B, H, N)}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"forward": _exact_forward, "backward": _exact_backward, "decode": _exact_decode, "evict": _exact_decode,
                "compact": _exact_compact}[case["op"]](s)
