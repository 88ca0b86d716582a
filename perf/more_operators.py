"""Timing cases of decoding over a paged cache of segment memories: its single-token step, the reads of a tree of drafted
tokens, the acceptance of one of its paths, forks of sequences that share pages, and the compaction of a pool.

A page holds one completed segment of one sequence, the memories of all its heads; a sequence's table names its pages in order
of time, and several tables may name the same page (``refs`` counts them, 0 is a free page).  What else a sequence has -- the
memory and key sum of its unfinished segment, its table and its position -- lies in a row of the cache, and ``row`` says
which row is whose.  ``run`` makes one pass, through the package where ``own`` is true and otherwise in plain torch
operations with the bookkeeping on the host; ``exact`` is the definition in 64 bits, token by token:

    e = v - a M k,  M <- a M + beta e k^T       (the gated delta memory; a = beta = 1 and e = v for the linear one)
    y = g_on M q + sum_i g_i M^(i) q            (gates as in the sequence's other operators)
"""
import copy
import random

import torch

own = False

RESIDUAL, GRM, SSC, MEAN = 0, 1, 3, 4


def listed():
    return [
        # one user of a small model, tokens one by one, over a segment's end: latency
        dict(name="step one user", op="step", B=1, H=4, d=64, C=64, n=5, mode=GRM, topk=0, dtype="bf16", delta=False, tokens=8),
        # a serving batch at unlike positions, each sequence a continuation that shares its prompt's pages
        dict(name="step batch ragged", op="step", B=8, H=16, d=128, C=256, n=63, mode=GRM, topk=0, dtype="bf16", delta=True, tokens=4),
        # one user, a short draft with two branches
        dict(name="tree one user", op="tree", B=1, H=4, d=64, C=64, n=5, T=7, shape="tree", mode=GRM, topk=0, dtype="bf16", delta=False),
        # a serving batch, a tree of 32 drafted tokens for every sequence
        dict(name="tree batch T32", op="tree", B=8, H=16, d=128, C=256, n=63, T=32, shape="tree", mode=GRM, topk=0, dtype="bf16", delta=False),
        # the widest draft over delta memories of long prompts
        dict(name="tree batch T64 delta", op="tree", B=12, H=16, d=128, C=512, n=96, T=64, shape="tree", mode=GRM, topk=0, dtype="bf16", delta=True),
        # full precision, the sparse router, short odd segments that the draft itself completes
        dict(name="tree f32 ssc odd", op="tree", B=3, H=6, d=64, C=7, n=29, T=13, shape="chain", mode=SSC, topk=3, dtype="f32", delta=True),
        # one user: the accepted path of a short draft
        dict(name="accept one user", op="accept", B=1, H=4, d=64, C=64, n=5, T=7, shape="tree", mode=GRM, topk=0, dtype="bf16", delta=False),
        # a serving batch: accepted paths of chains of 32, some over a segment's end
        dict(name="accept batch delta", op="accept", B=16, H=16, d=128, C=256, n=9, T=32, shape="chain", mode=GRM, topk=0, dtype="bf16", delta=True),
        # one prompt continued four times
        dict(name="fork four samples", op="fork", B=1, H=4, d=64, C=64, n=5, copies=4, dtype="bf16"),
        # four prompts continued eight times each, while as many finished sequences are freed
        dict(name="fork 4 prompts by 8", op="fork", B=4, H=16, d=128, C=256, n=63, copies=8, dtype="bf16"),
        # a small pool after some requests have left
        dict(name="compact small", op="compact", B=5, H=4, d=64, C=64, n=5, dtype="bf16"),
        # a large pool, half of it free, into one that fits
        dict(name="compact large", op="compact", B=12, H=16, d=128, C=512, n=48, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["step", "step", "tree", "tree", "tree", "accept", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 32, 16])
    case = dict(op=op, B=_log_int(rng, 1, 12), H=_log_int(rng, 1, 16), d=d, C=_log_int(rng, 3, 1024), n=_log_int(rng, 1, 90))
    if op == "fork":
        return case | dict(copies=_log_int(rng, 1, 8 if case["B"] < 5 else 2), dtype=dtype, B=min(case["B"], 8), n=min(case["n"], 63))
    if op == "compact":
        return case | dict(dtype=dtype, n=min(case["n"], 48))
    mode = rng.choice([GRM, GRM, GRM, SSC, SSC, MEAN, RESIDUAL])
    case |= dict(mode=mode, topk=rng.randint(1, 6) if mode == SSC else 0, dtype=dtype, delta=rng.random() < 0.5)
    if op == "step":
        return case | dict(tokens=rng.randint(1, 4), B=min(case["B"], 8), n=min(case["n"], 63))
    case |= dict(T=_log_int(rng, 1, 64 if dtype == "bf16" else 24), shape=rng.choice(["tree", "tree", "chain"]))
    if op == "accept":
        return case | dict(n=min(case["n"], 9))
    if dtype == "f32":
        case["B"] = min(case["B"], 4)
    return case


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------
NAMES = ("pages", "kbar", "refs", "online", "ksum", "table", "pos", "row")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _tokens(case, shape, kbar, g):
    """q, k, v, u [*shape, d] and log_alpha, beta [*shape]: each token asks for one of the sequence's topics ``kbar``
    [B, n, H, d] -- some far more often than others -- and its key is near another; shape is (B, H, ...)."""
    dev, t, d = "cuda", _dtype(case), case["d"]
    B, n, H = kbar.shape[:3]
    rnd = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    per = 1
    for x in shape[2:]:
        per *= x
    topics = _unit(kbar).permute(0, 2, 1, 3).reshape(B * H, n, d)

    def about():
        liked = torch.multinomial(torch.softmax(rnd(B * H, n), -1), per, replacement=True, generator=g)
        return torch.gather(topics, 1, liked[..., None].expand(-1, -1, d)).reshape(*shape, d)
    q, v = _unit(rnd(*shape, d)), rnd(*shape, d)
    k = _unit(0.7 * about() + rnd(*shape, d) * d ** -0.5)
    u = 4.0 * about() + rnd(*shape, d) * d ** -0.5
    la = -0.02 * torch.exp(rnd(*shape))
    be = torch.sigmoid(rnd(*shape))
    return [x.to(t).contiguous() for x in (q, k, v, u, la, be)]


def _draft(rng, T, shape):
    """Parents of T drafted tokens: a chain, or a tree whose likelier branches are deeper."""
    if shape == "chain":
        return list(range(-1, T - 1))
    return [-1 if j == 0 or rng.random() < 0.1 else max(rng.randrange(j), rng.randrange(j)) for j in range(T)]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    s = dict(case)
    op, B, H, d, C, n = (case[x] for x in ("op", "B", "H", "d", "C", "n"))
    rnd = lambda *x: torch.randn(*x, device="cuda", generator=g)  # noqa: E731
    ahead = case.get("tokens", case.get("T", 1))  # tokens that a pass may add to a sequence
    # sequences: prompts of up to n segments (the case says of how many), the longest n; half of them near a segment's end
    segs = [n] + [max(1, n - (7 * b + n * b // (2 * B)) % (n // 2 + 1)) for b in range(1, B)]
    part = [C - 1 - rng.randrange(min(C, ahead)) if rng.random() < 0.5 else rng.randrange(C) for _ in range(B)]
    per = {"step": 1, "accept": 1, "fork": case.get("copies", 0)}.get(op, 0)  # continuations of each prompt
    S = B + per * B
    adds = per * B * (ahead // C + 1) if op in ("step", "accept") else 0
    gone = sum(segs) if op == "compact" else n  # pages that no table names
    P = sum(segs) + adds + gone
    n_max = n + ahead // C + 1
    where = list(range(P))
    rng.shuffle(where)
    table = [[-1] * n_max for _ in range(S)]
    pos, row, refs = [0] * S, list(range(S)), [0] * P
    rng.shuffle(row)
    for b in range(B):
        pos[row[b]] = segs[b] * C + part[b]
        for i in range(segs[b]):
            p = where.pop()
            table[row[b]][i], refs[p] = p, 1
    if op == "fork":  # each continuation's slot holds a finished sequence, which shares the first prompt's pages
        for x in range(B, S):
            pos[row[x]] = segs[0] * C
            table[row[x]][:segs[0]] = table[row[0]][:segs[0]]
        for p in table[row[0]][:segs[0]]:
            refs[p] += S - B
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = {"pages": rnd(P, H, d, d) * 0.5, "kbar": _unit(rnd(P, H, d)) * 0.6, "online": rnd(S, H, d, d) * 0.3,
         "ksum": rnd(S, H, d) * 0.3, "refs": ints(refs), "table": ints(table), "pos": ints(pos), "row": ints(row)}
    if own:
        import memory_caching_linear_gb300 as mcl
        s["cache"] = mcl.PagedCache(S, H, d, C, n_max, P)
        for name in NAMES:
            getattr(s["cache"], name).copy_(c[name])
        if op == "compact":
            s["into"] = mcl.PagedCache(S, H, d, C, n_max, sum(segs))
        del c
        c = {name: getattr(s["cache"], name) for name in NAMES}
    else:
        s["host"] = {"refs": refs, "table": table, "pos": pos, "row": row}
    s["c"] = c
    if op == "compact":
        s["P"] = sum(segs)
        return s
    # which slot each slot goes on from: the prompts stay, the slots behind them are continuations (or free)
    s["src"] = [x if x < B else (x - B) % B if x < B + per * B else -1 for x in range(S)]
    s["src_dev"] = ints(s["src"])
    if op == "fork":
        return s
    if op == "tree":
        s["slots"] = rng.sample(range(B), B)
    else:
        s["slots"] = list(range(B, S))
    s["slots_dev"] = ints(s["slots"])
    first = [row[x] if op == "tree" else row[s["src"][x]] for x in s["slots"]]  # the row that a batch row goes on from
    some = min(segs)
    kbar = c["kbar"][torch.tensor([table[r][:some] for r in first], device="cuda")]
    R = len(first)
    if op == "step":
        s["toks"] = [_tokens(case, (R, H), kbar, g) for _ in range(case["tokens"])]
    else:
        T = case["T"]
        s["toks"] = _tokens(case, (R, H, T), kbar, g)
        s["count"] = [T] + [rng.randint(max(1, T // 2), T) for _ in range(R - 1)]
        s["parent"] = [_draft(rng, T, case["shape"]) for _ in range(R)]
        s["count_dev"], s["parent_dev"] = ints(s["count"]), ints(s["parent"])
        if op == "tree":
            s["y"] = torch.zeros(R, H, T, d, dtype=_dtype(case), device="cuda")  # drafts differ in length: the rest stays
        else:
            s["last"] = [rng.randrange(cnt) if rng.random() < 0.3 else cnt - 1 for cnt in s["count"]]
            s["last_dev"] = ints(s["last"])
    if case["mode"] in (RESIDUAL, MEAN):
        s["toks"] = [t[:3] + [None] + t[4:] for t in s["toks"]] if op == "step" else s["toks"][:3] + [None] + s["toks"][4:]
    return s


# ----------------------------------------------------------------------------------------------------------------
# the plain form: bookkeeping on the host, in 32 bits on the GPU (scores, which are ranked, in 64)
# ----------------------------------------------------------------------------------------------------------------
def _plain_fork(c, h, src):
    S, old = len(src), list(h["row"])
    keeper = {}
    for x in range(S):
        if src[x] >= 0 and (src[x] not in keeper or src[x] == x):
            keeper[src[x]] = x  # the slot itself if it stays, else the first that goes on from it
    kept = {x: old[f] for f, x in keeper.items()}
    spare = sorted(set(range(S)) - set(kept.values()))
    for x in range(S):
        if x in kept:
            h["row"][x] = kept[x]
            continue
        r = h["row"][x] = spare.pop(0)
        for p in h["table"][r]:
            if p >= 0:
                h["refs"][p] -= 1
        if src[x] < 0:
            h["table"][r], h["pos"][r] = [-1] * len(h["table"][r]), 0
            continue
        f = old[src[x]]
        c["online"][r].copy_(c["online"][f])
        c["ksum"][r].copy_(c["ksum"][f])
        h["table"][r], h["pos"][r] = list(h["table"][f]), h["pos"][f]
        for p in h["table"][r]:
            if p >= 0:
                h["refs"][p] += 1


def _books(c, h):
    for name in ("refs", "table", "pos", "row"):
        c[name] = torch.tensor(h[name], dtype=torch.int32, device="cuda")
    return {name: c[name] for name in NAMES}


def _held(h, r, C):
    """A row's completed segments that have a page."""
    return [p for p in h["table"][r][:h["pos"][r] // C] if p >= 0]


def _weights(r, ready, mode, topk):
    """Gates over [..., memories] whose last is the online one; the others count where ``ready``."""
    ok = torch.cat([ready, torch.ones_like(ready[..., :1])], -1)
    if mode == RESIDUAL:
        return ok.float()
    if mode == MEAN:
        return ok.float() / ok.sum(-1, keepdim=True)
    r = r.masked_fill(~ok, float("-inf"))
    if mode == SSC:
        rank = torch.argsort(torch.argsort(r[..., :-1], dim=-1, descending=True, stable=True), -1)
        r = torch.cat([r[..., :-1].masked_fill(rank >= topk, float("-inf")), r[..., -1:]], -1)
    w = torch.exp(r - r.amax(-1, keepdim=True))
    return (w / w.sum(-1, keepdim=True)).float()


def _advance(s, c, h, r, k, v, la, be):
    """One token of row r: k, v [H, d], la, be [H]."""
    C, M, ks = s["C"], c["online"][r], c["ksum"][r]
    k, v = k.float(), v.float()
    if h["pos"][r] % C == 0:
        M.zero_()
        ks.zero_()
    if s["delta"]:
        M.mul_(torch.exp(la.float())[:, None, None])
        v = be.float()[:, None] * (v - (M @ k[..., None])[..., 0])
    M.add_(v[..., None] * k[:, None])
    ks.add_(k)
    h["pos"][r] += 1


def _complete(s, c, h, r):
    """The row's segment that has just ended goes to the page that was set aside for it."""
    p = h["table"][r][h["pos"][r] // s["C"] - 1]
    c["pages"][p].copy_(c["online"][r])
    c["kbar"][p].copy_(c["ksum"][r] / s["C"])


def _set_aside(h, r, segments, C):
    for _ in range(segments):
        p = h["refs"].index(0)
        h["table"][r][h["table"][r].index(-1)], h["refs"][p] = p, 1


def _plain_step(s, c, h, tok):
    C, mode = s["C"], s["mode"]
    out = torch.empty_like(tok[0])
    rows = [h["row"][x] for x in s["slots"]]
    for r in rows:
        _set_aside(h, r, (h["pos"][r] + 1) // C - h["pos"][r] // C, C)
    for b, r in enumerate(rows):
        q, k, v, u, la, be = (None if x is None else x[b] for x in tok)
        held = _held(h, r, C)
        _advance(s, c, h, r, k, v, la, be)
        M = c["pages"][held]  # [n, H, d, d]
        score = None
        if u is not None:
            cached = torch.einsum("nhd,hd->hn", c["kbar"][held].double(), u.double())
            online = (u.double() * c["ksum"][r].double()).sum(-1) / ((h["pos"][r] - 1) % C + 1)
            score = torch.cat([cached, online[:, None]], -1)
        w = _weights(score, torch.ones(s["H"], len(held), dtype=torch.bool, device=q.device), mode, s["topk"])
        qf = q.float()
        read = (M @ qf[None, ..., None])[..., 0]  # [n, H, d]
        y = w[:, -1:] * (c["online"][r] @ qf[..., None])[..., 0] + torch.einsum("hn,nhd->hd", w[:, :-1], read)
        out[b] = y.to(out.dtype)
        if h["pos"][r] % C == 0:
            _complete(s, c, h, r)
    return out


def _plain_tree(s, c, h):
    C, mode, T, H = s["C"], s["mode"], s["T"], s["H"]
    for b, x in enumerate(s["slots"]):
        r, m = h["row"][x], s["count"][b]
        q, k, v, u, la, be = (None if z is None else z[b, :, :m].float() for z in s["toks"])  # [H, m, d], [H, m]
        dev = q.device
        pos, held, parent = h["pos"][r], _held(h, r, C), s["parent"][b][:m]
        anc = [[False] * m for _ in range(m)]
        depth = [0] * m
        for j, f in enumerate(parent):
            if f >= 0:
                anc[j], depth[j] = list(anc[f]), depth[f] + 1
            anc[j][j] = True
        seg = [(pos % C + e) // C for e in depth]  # 0 is the segment that the cache has begun
        J = max(seg) + 1
        anc, seg, depth = (torch.tensor(z, device=dev) for z in (anc, seg, depth))
        of = anc[:, None] & (seg[None, None] == torch.arange(J, device=dev)[None, :, None])  # [node, segment, ancestor]
        own_seg = torch.gather(of, 1, seg[:, None, None].expand(m, 1, m))[:, 0]  # ancestors of the node's own segment
        begun = pos % C > 0
        M0 = c["online"][r] if begun else torch.zeros_like(c["online"][r])
        # gates: cached memories, then the path's segments 0 .. J-1 (the node's own one is the online memory)
        score, n = None, len(held)
        is_on = torch.arange(J, device=dev)[None] == seg[:, None]
        past = torch.arange(J, device=dev)[None] < seg[:, None]
        if u is not None:
            ud = u.double()
            cached = torch.einsum("nhd,hmd->hmn", c["kbar"][held].double(), ud)
            path = torch.einsum("hma,mja->hmj", ud @ k.double().transpose(1, 2), of.double())
            if begun:
                path[..., 0] += (ud * c["ksum"][r].double()[:, None]).sum(-1)
            length = torch.where(is_on, ((pos + depth) % C + 1)[:, None], C)
            path = path / length
            online = torch.gather(path, 2, seg[None, :, None].expand(H, m, 1))
            score = torch.cat([cached, path, online], -1)
        ready = torch.cat([torch.ones(m, n, dtype=torch.bool, device=dev), past], -1).expand(H, m, n + J)
        w = _weights(score, ready, mode, s["topk"])
        w_path = torch.where(is_on, w[..., -1:], w[..., n:n + J])  # [H, m, J]
        y = torch.zeros(H, m, s["d"], device=dev)
        for i, p in enumerate(held):
            y += w[..., i:i + 1] * (q @ c["pages"][p].transpose(1, 2))
        # the memory of segment j as node x sees it: decay . M0 (j = 0) and what x's ancestors in j wrote
        if s["delta"]:
            cum = torch.einsum("ma,ha->hm", own_seg.double(), la.double())  # of each node within its segment
            last = torch.where(of, torch.arange(m, device=dev), -1).amax(-1)  # [node, segment]: the deepest ancestor
            decay = torch.exp(cum[:, last.clamp_min(0)][..., seg] - cum[:, None]).float()  # [H, node, ancestor]
            into0 = torch.exp(cum[:, last[:, 0].clamp_min(0)]).float()
            near = own_seg & ~torch.eye(m, dtype=torch.bool, device=dev)
            kk = (k @ k.transpose(1, 2)) * torch.where(near, decay * be[:, None], 0.0)
            e = v - torch.where((seg == 0)[:, None], into0[..., None] * (k @ M0.transpose(1, 2)), 0.0)
            for j in range(1, m):
                e[:, j] -= (kk[:, j, None, :j] @ e[:, :j])[:, 0]
            write = be[..., None] * e
        else:
            decay, into0, write = torch.ones(H, m, m, device=dev), torch.ones(H, m, device=dev), v
        g_anc = w_path[..., seg] * torch.where(anc, decay, 0.0)
        y += (g_anc * (q @ k.transpose(1, 2))) @ write + (w_path[..., 0] * into0)[..., None] * (q @ M0.transpose(1, 2))
        s["y"][b, :, :m] = y.to(s["y"].dtype)
    return s["y"]


def _path(parent, last):
    out = []
    while last >= 0:
        out.append(last)
        last = parent[last]
    return out[::-1]


def _plain_accept(s, c, h):
    C = s["C"]
    rows = [h["row"][x] for x in s["slots"]]
    paths = [_path(s["parent"][b], s["last"][b]) for b in range(len(rows))]
    for r, path in zip(rows, paths):
        _set_aside(h, r, (h["pos"][r] + len(path)) // C - h["pos"][r] // C, C)
    for b, (r, path) in enumerate(zip(rows, paths)):
        for j in path:
            _, k, v, _, la, be = (None if x is None else x[b, :, j] for x in s["toks"])
            _advance(s, c, h, r, k, v, la, be)
            if h["pos"][r] % C == 0:
                _complete(s, c, h, r)


def _plain_compact(s, c, h):
    live = [p for p in range(len(h["refs"])) if h["refs"][p] > 0]
    to = {p: i for i, p in enumerate(live)} | {-1: -1}
    S, dev = len(h["row"]), c["pages"].device
    at = torch.tensor(live, device=dev)
    got = {"pages": c["pages"][at], "kbar": c["kbar"][at], "refs": [h["refs"][p] for p in live],
           "online": c["online"][h["row"]], "ksum": c["ksum"][h["row"]],
           "table": [[to[p] for p in h["table"][r]] for r in h["row"]], "pos": [h["pos"][r] for r in h["row"]],
           "row": list(range(S))}
    return {n: torch.tensor(x, dtype=torch.int32, device=dev) if isinstance(x, list) else x for n, x in got.items()}


def run(s):
    op = s["op"]
    if own:
        import memory_caching_linear_gb300 as mcl
        c = s["cache"]
        if op == "compact":
            mcl.mc_pages_compact(s["into"], c)
            return {name: getattr(s["into"], name) for name in NAMES}
        if op == "tree":
            q, k, v, u, la, be = s["toks"]
            gated = dict(log_alpha=la, beta=be) if s["delta"] else {}
            return mcl.mc_decode_tree(c, q, k, v, u, s["parent_dev"], s["mode"], s["topk"], count=s["count_dev"],
                                      slots=s["slots_dev"], y=s["y"], **gated)
        mcl.mc_pages_fork(c, s["src_dev"])  # the continuations begin at their prompts (again)
        got = {}
        if op == "step":
            got["y"] = [mcl.mc_decode_step_paged(c, q, k, v, u, s["mode"], s["topk"], slots=s["slots_dev"],
                                                 **(dict(log_alpha=la, beta=be) if s["delta"] else {}))
                        for q, k, v, u, la, be in s["toks"]]
        elif op == "accept":
            _, k, v, _, la, be = s["toks"]
            gated = dict(log_alpha=la, beta=be) if s["delta"] else {}
            mcl.mc_tree_accept(c, k, v, s["parent_dev"], s["last_dev"], slots=s["slots_dev"], **gated)
        return got | {name: getattr(c, name) for name in NAMES}
    c, h = s["c"], s["host"]
    if op == "compact":
        return _plain_compact(s, c, h)
    if op == "tree":
        return _plain_tree(s, c, h)
    _plain_fork(c, h, s["src"])
    got = {}
    if op == "step":
        got["y"] = [_plain_step(s, c, h, tok) for tok in s["toks"]]
    elif op == "accept":
        _plain_accept(s, c, h)
    return got | _books(c, h)


# ----------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    op, B, H, d, C, n = (case[x] for x in ("op", "B", "H", "d", "C", "n"))
    e = 2 if case["dtype"] == "bf16" else 4
    state = H * (4 * d * d)  # a page, or a row's memory
    segs = n + (B - 1) * (max(1, n // 2) + n) / 2  # the prompts' pages, on average
    if op == "compact":
        return {"bytes": int(2 * segs * (state + 4 * H * d) + 2 * B * state), "flops": 0}
    if op == "fork":
        return {"bytes": int((B + B * (case["copies"])) * state), "flops": 0}
    vals = H * d * e * (4 if case["mode"] in (GRM, SSC) else 3)
    if op == "accept":  # the continuation's memory is read from its prompt's and written once
        mean = 0.85 * case["T"] * 0.75
        return {"bytes": int(B * (2 * state + mean * 2 * H * d * e + mean / C * state)), "flops": int(B * H * mean * 4 * d * d)}
    T = case.get("tokens", case.get("T"))
    need = min(1.0, case["topk"] * (T if op == "tree" else 1) / n) if case["mode"] == SSC else 1.0  # pages that a gate weighs
    if op == "tree":
        live = 1 + (B - 1) * 0.75 if B > 1 else 1
        return {"bytes": int(segs * (need * state + 4 * H * d) + B * state + live * T * (vals + H * d * e)),
                "flops": int(T * 2 * H * d * d * (segs * (need if case["mode"] != SSC else min(1.0, case["topk"] / n)) + B * (2 if case["delta"] else 1)))}
    return {"bytes": int(T * (segs * (need * state + 4 * H * d) + B * (2 * state + vals + H * d * e))),
            "flops": int(T * 2 * H * d * d * (segs * need + 4 * B))}


# ----------------------------------------------------------------------------------------------------------------
# the definition, token by token, in 64 bits
# ----------------------------------------------------------------------------------------------------------------
class _Sequence:
    """One sequence: completed segments' memories [n, H, d, d] and mean keys [n, H, d], those of the tokens that it took itself
    (``new``), the online memory and key sum."""

    def __init__(self, memories, means, online, total, pos, C):
        self.memories, self.means, self.new, self.C, self.pos = memories, means, [], C, pos
        self.M, self.total = online, total

    def taken(self, k, v, la, be):
        """The sequence with one more token (this one stays as it is)."""
        s = copy.copy(self)
        M, total = (self.M, self.total) if self.pos % self.C else (torch.zeros_like(self.M), torch.zeros_like(self.total))
        if la is not None:
            M = la.exp()[:, None, None] * M
            v = be[:, None] * (v - torch.einsum("hij,hj->hi", M, k))
        s.M, s.total = M + torch.einsum("hi,hj->hij", v, k), total + k
        s.pos = self.pos + 1
        return s

    def closed(self):
        """What follows a token: a full segment joins the completed ones."""
        if self.pos % self.C == 0:
            self.new = self.new + [(self.M, self.total / self.C)]
        return self

    def read(self, q, u, mode, topk):
        """y [H, d] of the token that was just taken."""
        n = self.memories.shape[0]
        reads = [torch.einsum("nhij,hj->nhi", self.memories, q)] + [torch.einsum("hij,hj->hi", M, q)[None] for M, _ in self.new]
        reads = torch.cat(reads)  # [all, H, d]
        on = torch.einsum("hij,hj->hi", self.M, q)
        total = len(reads)
        if mode in (RESIDUAL, MEAN):
            return (on + reads.sum(0)) / (1 if mode == RESIDUAL else total + 1)
        r = [torch.einsum("nhj,hj->nh", self.means, u)] + [torch.einsum("hj,hj->h", z, u)[None] for _, z in self.new]
        r = torch.cat(r).T  # [H, all]
        if mode == SSC and topk < total:
            best = torch.sort(r, dim=-1, descending=True, stable=True).indices[:, :topk]
            r = torch.full_like(r, float("-inf")).scatter(1, best, torch.gather(r, 1, best))
        r_on = (u * self.total).sum(-1, keepdim=True) / ((self.pos - 1) % self.C + 1)
        w = torch.softmax(torch.cat([r, r_on], -1), -1)
        return torch.einsum("hn,nhi->hi", w[:, :-1], reads) + w[:, -1:] * on


def _sequence(s, books, r):
    c, C = s["c"], s["C"]
    pages = [p for p in books["table"][r][:books["pos"][r] // C] if p >= 0]
    return _Sequence(c["pages"][pages].double(), c["kbar"][pages].double(), c["online"][r].double(), c["ksum"][r].double(),
                     books["pos"][r], C)


def _exact_books(s):
    return {name: s["c"][name].tolist() for name in ("refs", "table", "pos", "row")}


def _exact_forked(s, books):
    """Rows after the fork, and for every row that is written the row it is copied from (-1: freed)."""
    src, old = s["src"], list(books["row"])
    S, new, taken = len(src), [-1] * len(src), set()
    for f in range(S):
        heirs = [x for x in range(S) if src[x] == f]
        if heirs:
            x = f if f in heirs else heirs[0]
            new[x] = old[f]
            taken.add(old[f])
    spare = iter(r for r in range(S) if r not in taken)
    copied = {}
    for x in range(S):
        if new[x] < 0:
            new[x] = next(spare)
            copied[new[x]] = old[src[x]] if src[x] >= 0 else -1
    table, pos = [list(t) for t in books["table"]], list(books["pos"])
    for r, f in copied.items():
        table[r] = list(books["table"][f]) if f >= 0 else [-1] * len(table[r])
        pos[r] = books["pos"][f] if f >= 0 else 0
    refs = [0] * len(books["refs"])
    for t in table:
        for p in t:
            if p >= 0:
                refs[p] += 1
    return {"refs": refs, "table": table, "pos": pos, "row": new}, copied


def exact(case, seed):
    s = prepare(case, seed)
    c, C, op = s["c"], s["C"], s["op"]
    books = _exact_books(s)
    as_tensor = lambda b: {n: torch.tensor(b[n], dtype=torch.int32, device="cuda") for n in b}  # noqa: E731
    if op == "compact":
        live = [p for p, x in enumerate(books["refs"]) if x]
        rows = books["row"]
        table = [[live.index(p) if p >= 0 else -1 for p in books["table"][r]] for r in rows]
        return {"pages": c["pages"][live].double(), "kbar": c["kbar"][live].double(), "online": c["online"][rows].double(),
                "ksum": c["ksum"][rows].double()} | as_tensor({"refs": [books["refs"][p] for p in live], "table": table,
                                                               "pos": [books["pos"][r] for r in rows], "row": list(range(len(rows)))})
    gated = (lambda la, be: (la, be)) if case.get("delta") else (lambda la, be: (None, None))
    wide = lambda x: None if x is None else x.double()  # noqa: E731
    if op == "tree":
        out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for b, x in enumerate(s["slots"]):
            root, nodes = _sequence(s, books, books["row"][x]), []
            q, k, v, u, la, be = (wide(None if z is None else z[b]) for z in s["toks"])
            for j in range(s["count"][b]):
                f = s["parent"][b][j]
                now = (nodes[f] if f >= 0 else root).taken(k[:, j], v[:, j], *gated(la[:, j], be[:, j]))
                out[b, :, j] = now.read(q[:, j], None if u is None else u[:, j], s["mode"], s["topk"])
                nodes.append(now.closed())
        return out
    after, copied = _exact_forked(s, books)
    big = {n: c[n].double() for n in ("pages", "kbar", "online", "ksum")}
    for n in ("online", "ksum"):
        whole = big[n].clone()
        for r, f in copied.items():
            if f >= 0:
                whole[r] = big[n][f]
        big[n] = whole
    got = {}
    if op != "fork":
        rows = [after["row"][x] for x in s["slots"]]
        seqs = {}
        for b, r in enumerate(rows):
            pages = [p for p in after["table"][r][:after["pos"][r] // C] if p >= 0]
            seqs[b] = _Sequence(big["pages"][pages], big["kbar"][pages], big["online"][r], big["ksum"][r], after["pos"][r], C)
        turns = s["tokens"] if op == "step" else 1
        ys = [[] for _ in range(turns)]
        for turn in range(turns):
            for b, r in enumerate(rows):
                if op == "step":
                    todo = [[wide(None if z is None else z[b]) for z in s["toks"][turn]]]
                else:
                    todo, j = [], s["last"][b]
                    while j >= 0:
                        todo.insert(0, [wide(None if z is None else z[b, :, j]) for z in s["toks"]])
                        j = s["parent"][b][j]
                for q, k, v, u, la, be in todo:
                    seqs[b] = seqs[b].taken(k, v, *gated(la, be))
                    if op == "step":
                        ys[turn].append(seqs[b].read(q, u, s["mode"], s["topk"]))
                    had = len(seqs[b].new)
                    seqs[b].closed()
                    if len(seqs[b].new) > had:
                        p = after["refs"].index(0)
                        after["refs"][p] = 1
                        after["table"][r][seqs[b].pos // C - 1] = p
                        big["pages"][p], big["kbar"][p] = seqs[b].new[-1]
        for b, r in enumerate(rows):
            big["online"][r], big["ksum"][r], after["pos"][r] = seqs[b].M, seqs[b].total, seqs[b].pos
        if op == "step":
            got["y"] = [torch.stack(y) for y in ys]
    return got | big | as_tensor(after)
