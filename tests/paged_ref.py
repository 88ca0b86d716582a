"""A paged cache and its operators in 64 bits on the CPU, token by token, with the same rules for pages, rows and bad indexes
as mc.h gives: what the GPU tests compare with."""
import random

import torch

RESIDUAL, GRM, SOUP, SSC, MEAN = 0, 1, 2, 3, 4
INDEX, NONE_FREE, TABLE_FULL = 1, 2, 4
FLOATS, INTS = ("pages", "kbar", "online", "ksum"), ("refs", "table", "pos", "row", "status")


def read(memories, means, M, mean_on, q, u, mode, topk):
    """y [H, d] over completed memories (lists of [H, d, d] and [H, d]) and the online one."""
    H, d = q.shape
    on = torch.einsum("hij,hj->hi", M, q)
    n = len(memories)
    if n == 0:
        return on
    got = torch.stack([torch.einsum("hij,hj->hi", m, q) for m in memories])  # [n, H, d]
    if mode in (RESIDUAL, MEAN):
        return (on + got.sum(0)) / (1 if mode == RESIDUAL else n + 1)
    out = torch.zeros(H, d, dtype=torch.float64)
    for h in range(H):
        r = torch.stack([means[i][h] @ u[h] for i in range(n)])
        take = list(range(n))
        if mode == SSC:
            # scores are ranked as the fp32 numbers that the router forms; equal ones: the older
            take = sorted(range(n), key=lambda i: (-float(r[i].float()), i))[:topk]
        z = torch.cat([r[take], (mean_on[h] @ u[h])[None]])
        w = torch.softmax(z, 0)
        out[h] = w[-1] * on[h]
        for x, i in enumerate(take):
            out[h] += w[x] * got[i, h]
    return out


class Ref:
    def __init__(self, S, H, d, C, n_max, P):
        self.S, self.H, self.d, self.C, self.n_max, self.P = S, H, d, C, n_max, P
        f = dict(dtype=torch.float64)
        self.pages, self.kbar = torch.zeros(P, H, d, d, **f), torch.zeros(P, H, d, **f)
        self.online, self.ksum = torch.zeros(S, H, d, d, **f), torch.zeros(S, H, d, **f)
        self.refs, self.table = [0] * P, [[-1] * n_max for _ in range(S)]
        self.pos, self.row, self.status = [0] * S, list(range(S)), [0]

    def to(self, cache):
        """Into a PagedCache."""
        for n in FLOATS + INTS:
            x = getattr(self, n)
            getattr(cache, n).copy_(x if torch.is_tensor(x) else torch.tensor(x))
        return cache

    def fill(self, segs, part, gen, rng):
        """Prompts of segs[x] segments and part[x] tokens, on pages in no order."""
        free = [p for p in range(self.P) if self.refs[p] == 0]
        rng.shuffle(free)
        r32 = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731 (fp32 numbers: what the GPU starts from)
        self.pages[:], self.kbar[:] = r32(*self.pages.shape) * 0.5, r32(*self.kbar.shape) * 0.5
        self.online[:], self.ksum[:] = r32(*self.online.shape) * 0.3, r32(*self.ksum.shape) * 0.3
        for x, (n, m) in enumerate(zip(segs, part)):
            r = self.row[x]
            self.pos[r] = n * self.C + m
            for i in range(n):
                self.table[r][i] = free.pop()
                self.refs[self.table[r][i]] = 1
        return self

    # ---- rules
    def act(self, slots, B, writes):
        rows, seen = [], set()
        for b in range(B):
            x = b if slots is None else slots[b]
            if x == -1:
                rows.append(None)
            elif not 0 <= x < self.S or (writes and x in seen):
                self.status[0] |= INDEX
                rows.append(None)
            else:
                seen.add(x)
                rows.append(self.row[x])
        return rows

    def take(self, r, s0, s1):
        """Pages for segments s0 .. s1 - 1 of row r."""
        for s in range(s0, s1):
            if s >= self.n_max:
                self.status[0] |= TABLE_FULL
                continue
            p = next((p for p in range(self.P) if self.refs[p] == 0), -1)
            if p < 0:
                self.status[0] |= NONE_FREE
            else:
                self.refs[p] = 1
            self.table[r][s] = p

    def held(self, r):
        return [p for p in self.table[r][:min(self.pos[r] // self.C, self.n_max)] if p >= 0]

    @staticmethod
    def token(M, ks, pos, C, k, v, la, be):
        if pos % C == 0:
            M, ks = torch.zeros_like(M), torch.zeros_like(ks)
        if la is not None:
            M = la.clamp_min(-60).exp()[:, None, None] * M
            v = be[:, None] * (v - torch.einsum("hij,hj->hi", M, k))
        return M + torch.einsum("hi,hj->hij", v, k), ks + k

    # ---- operators (q, k, v, u [B, H, (T,) d] in any dtype)
    def tree(self, q, k, v, u, la, be, parent, count, slots, mode, topk):
        """{(b, node): y [H, d]}"""
        B, _, T, _ = q.shape
        out = {}
        for b, r in enumerate(self.act(slots, B, False)):
            if r is None:
                continue
            m = T if count is None else min(max(count[b], 0), T)
            if count is not None and m != count[b]:
                self.status[0] |= INDEX
            base = self.held(r)
            states = []  # per node: memory, key sum, position after it, what its path completed
            for j in range(m):
                f = parent[b][j]
                if not -1 <= f < j:
                    self.status[0] |= INDEX
                    f = -1
                M, ks, pos, new = states[f] if f >= 0 else (self.online[r], self.ksum[r], self.pos[r], [])
                g = (None, None) if la is None else (la[b, :, j].double(), be[b, :, j].double())
                M, ks = self.token(M, ks, pos, self.C, k[b, :, j].double(), v[b, :, j].double(), *g)
                pos += 1
                mem = [self.pages[p] for p in base] + [x[0] for x in new]
                mean = [self.kbar[p] for p in base] + [x[1] for x in new]
                out[b, j] = read(mem, mean, M, ks / ((pos - 1) % self.C + 1), q[b, :, j].double(),
                                 None if u is None else u[b, :, j].double(), mode, topk)
                states.append((M, ks, pos, new + [(M, ks / self.C)] if pos % self.C == 0 else new))
        return out

    def accept(self, k, v, la, be, parent, last, slots):
        B, _, T, _ = k.shape
        rows, paths = self.act(slots, B, True), []
        for b in range(B):
            path, x = [], last[b]
            if not -1 <= x < T:
                self.status[0] |= INDEX
                x = -1
            while x >= 0:
                path.insert(0, x)
                f = parent[b][x]
                if not -1 <= f < x:
                    self.status[0] |= INDEX
                    f = -1
                x = f
            paths.append(path)
        for r, path in zip(rows, paths):
            if r is not None:
                self.take(r, self.pos[r] // self.C, (self.pos[r] + len(path)) // self.C)
        for b, (r, path) in enumerate(zip(rows, paths)):
            for j in path if r is not None else []:
                g = (None, None) if la is None else (la[b, :, j].double(), be[b, :, j].double())
                self.advance(r, k[b, :, j].double(), v[b, :, j].double(), *g)

    def advance(self, r, k, v, la, be):
        self.online[r], self.ksum[r] = self.token(self.online[r], self.ksum[r], self.pos[r], self.C, k, v, la, be)
        self.pos[r] += 1
        s = self.pos[r] // self.C - 1
        if self.pos[r] % self.C == 0 and s < self.n_max and self.table[r][s] >= 0:
            self.pages[self.table[r][s]], self.kbar[self.table[r][s]] = self.online[r], self.ksum[r] / self.C

    def step(self, q, k, v, u, la, be, slots, mode, topk):
        add = lambda x: None if x is None else x[:, :, None]  # noqa: E731
        rows = self.act(slots, q.shape[0], True)
        own = [x if r is not None else -1 for x, r in zip(slots or range(q.shape[0]), rows)]
        none = [[-1]] * q.shape[0]
        out = self.tree(*(add(x) for x in (q, k, v, u, la, be)), none, None, own, mode, topk)
        self.accept(add(k), add(v), add(la), add(be), none, [0] * q.shape[0], own)
        return {b: y for (b, _), y in out.items()}

    def fork(self, src):
        old = list(self.row)
        f = [x if not -1 <= s < self.S else s for x, s in enumerate(src)]
        if f != list(src):
            self.status[0] |= INDEX
        heir = {}
        for x in range(self.S):
            if f[x] >= 0 and (f[x] not in heir or f[x] == x):
                heir[f[x]] = x
        stays = {x: old[s] for s, x in heir.items()}
        spare = sorted(set(range(self.S)) - set(stays.values()))
        for x in range(self.S):
            if x in stays:
                self.row[x] = stays[x]
                continue
            r = self.row[x] = spare.pop(0)
            if f[x] < 0:
                self.table[r], self.pos[r] = [-1] * self.n_max, 0
            else:
                o = old[f[x]]
                self.online[r], self.ksum[r] = self.online[o], self.ksum[o]
                self.table[r], self.pos[r] = list(self.table[o]), self.pos[o]
        self.recount()

    def recount(self):
        self.refs = [0] * self.P
        for t in self.table:
            for p in t:
                if p >= 0:
                    self.refs[p] += 1

    def compact(self, S, n_max, P):
        to = Ref(S, self.H, self.d, self.C, n_max, P)
        live = [p for p in range(self.P) if self.refs[p]]
        if len(live) > P:
            to.status[0] |= NONE_FREE
        where = {p: i if i < P else -1 for i, p in enumerate(live)} | {-1: -1}
        for p in live[:P]:
            to.pages[where[p]], to.kbar[where[p]], to.refs[where[p]] = self.pages[p], self.kbar[p], self.refs[p]
        for x in range(self.S):
            r = self.row[x]
            to.online[x], to.ksum[x], to.pos[x] = self.online[r], self.ksum[r], self.pos[r]
            to.table[x][:self.n_max] = [where[p] for p in self.table[r]]
        return to

    def load(self, slot, k, states):
        """k [H, L, d], states [H, N, d, d]"""
        r, L, C = self.row[slot], k.shape[1], self.C
        self.table[r], self.pos[r] = [-1] * self.n_max, 0
        self.recount()
        self.take(r, 0, L // C)
        self.pos[r] = L
        for i in range(L // C):
            p = self.table[r][i]
            if p >= 0:
                self.pages[p], self.kbar[p] = states[:, i].double(), k[:, i * C:(i + 1) * C].double().mean(1)
        tail = L % C
        self.online[r] = states[:, -1].double() if tail else 0.0
        self.ksum[r] = k[:, L - tail:].double().sum(1)


def draft(rng, B, T, shape):
    def one():
        if shape == "chain":
            return list(range(-1, T - 1))
        if shape == "star":
            return [-1] * T
        return [-1 if j == 0 or rng.random() < 0.15 else max(rng.randrange(j), rng.randrange(j)) for j in range(T)]
    return [one() for _ in range(B)]


def tokens(gen, B, H, T, d, dtype):
    """q, k, v, u, log_alpha, beta of a draft."""
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = [unit(r(B, H, T, d)), unit(r(B, H, T, d)), r(B, H, T, d), 2 * r(B, H, T, d), -0.1 * torch.exp(r(B, H, T)),
         2 * torch.sigmoid(r(B, H, T))]
    return [t.to(dtype) for t in x]


def seeded(seed):
    return torch.Generator().manual_seed(seed), random.Random(seed)
