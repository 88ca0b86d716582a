"""The 64-bit paged cache against itself: a tree's reads are those of steps along each path, and the bookkeeping holds."""
import copy

import pytest
import torch

from paged_ref import GRM, MEAN, RESIDUAL, SSC, Ref, draft, seeded, tokens


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2), (MEAN, 0), (RESIDUAL, 0)])
@pytest.mark.parametrize("C", [1, 3, 8])
@pytest.mark.parametrize("delta", [False, True])
def test_a_path_is_steps(C, delta, mode, topk):
    gen, rng = seeded(C)
    T, H, d = 7, 2, 16
    ref = Ref(2, H, d, C, 12, 30).fill([3, 0], [C // 2, 0], gen, rng)
    x = tokens(gen, 2, H, T, d, torch.float64)
    if not delta:
        x[4] = x[5] = None
    parent = draft(rng, 2, T, "tree")
    got = ref.tree(*x, parent, None, None, mode, topk)
    for b in range(2):
        for j in range(T):
            path, n = [], j
            while n >= 0:
                path.insert(0, n)
                n = parent[b][n]
            one = copy.deepcopy(ref)
            for n in path:
                y = one.step(*(None if t is None else t[b:b + 1, :, n] for t in x), [b], mode, topk)[0]
            assert (y - got[b, j]).abs().max() < 1e-12
            both = copy.deepcopy(ref)
            both.accept(x[1][b:b + 1], x[2][b:b + 1], *(None if t is None else t[b:b + 1] for t in x[4:]), parent[b:b + 1], [j], [b])
            assert torch.equal(both.pages, one.pages) and both.table == one.table and both.refs == one.refs and both.pos == one.pos


def test_forks_keep_what_they_go_on_from():
    gen, rng = seeded(5)
    ref = Ref(6, 1, 16, 4, 6, 24).fill([2, 1, 3, 0, 2, 0], [0, 1, 2, 3, 0, 0], gen, rng)
    for _ in range(30):
        old = copy.deepcopy(ref)
        src = [rng.randrange(-1, 6) for _ in range(6)]
        ref.fork(src)
        assert sorted(ref.row) == list(range(6))
        for x, f in enumerate(src):
            r, o = ref.row[x], old.row[f]
            assert ref.pos[r] == (old.pos[o] if f >= 0 else 0) and ref.table[r] == (old.table[o] if f >= 0 else [-1] * 6)
            if f >= 0:
                assert torch.equal(ref.online[r], old.online[o]) and torch.equal(ref.ksum[r], old.ksum[o])
