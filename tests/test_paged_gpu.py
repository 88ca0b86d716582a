"""The paged cache's operators on the GPU against their 64-bit forms, and together as a server uses them.

Tolerances, of an output's largest value, are those that mc.h gives: 1e-4 with fp32 inputs, 1e-2 with bf16 ones.  What is copied or
counted is equal."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from paged_ref import FLOATS, GRM, INDEX, INTS, MEAN, NONE_FREE, RESIDUAL, SOUP, SSC, TABLE_FULL, Ref, draft, seeded, tokens

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 1e-4, torch.bfloat16: 1e-2}
i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
gpu = lambda x: None if x is None else x.cuda()  # noqa: E731


def on_gpu(ref):
    return ref.to(mcl.PagedCache(ref.S, ref.H, ref.d, ref.C, ref.n_max, ref.P))


def near(got, want, tol):
    assert torch.isfinite(got).all()
    top = want.abs().max().clamp_min(1e-30)
    assert float((got.double().cpu() - want).abs().max() / top) <= tol


def same(cache, ref, tol=1e-4):
    for n in INTS:
        assert getattr(cache, n).cpu().tolist() == getattr(ref, n), n
    for n in FLOATS:
        got, want = getattr(cache, n).double().cpu(), getattr(ref, n)
        assert float((got - want).abs().max()) <= tol * float(want.abs().max().clamp_min(1.0)), n


def run_tree(cache, ref, x, parent, count, slots, mode, topk, dtype):
    B, H, T, d = x[0].shape
    y = torch.full((B, H, T, d), 7.0, dtype=dtype, device="cuda")
    q, k, v, u, la, be = (gpu(t) for t in x)
    mcl.mc_decode_tree(cache, q, k, v, u, i32(parent), mode, topk, log_alpha=la, beta=be, count=i32(count), slots=i32(slots), y=y)
    want = ref.tree(*x, parent, count, slots, mode, topk)
    got, ref_y = y.float().cpu(), torch.full((B, H, T, d), 7.0, dtype=torch.float64)
    for (b, j), z in want.items():
        ref_y[b, :, j] = z
    assert torch.isfinite(got).all()
    for b in range(B):
        rows = [j for (bb, j) in want if bb == b]
        rest = [j for j in range(T) if j not in rows]
        assert (got[b][:, rest] == 7.0).all()
        if rows:
            near(got[b][:, rows], ref_y[b][:, rows], TOL[dtype])
    assert cache.status.tolist() == ref.status
    return y


CASES = [  # d, H, C, T, shape, segments of each slot, tokens begun
    (16, 1, 5, 1, "chain", [3], [2]),
    (16, 3, 1, 9, "tree", [4, 0, 2], [0, 0, 0]),
    (32, 2, 7, 5, "tree", [2, 3], [6, 0]),
    (64, 2, 16, 8, "star", [5, 1, 0, 9], [15, 1, 0, 7]),
    (64, 3, 4, 33, "chain", [7, 2], [3, 0]),
    (128, 2, 64, 13, "tree", [4, 4, 1], [60, 0, 63]),
    (128, 1, 9, 64, "chain", [11], [4]),
    (64, 2, 100, 64, "tree", [1, 6, 3], [99, 40, 0]),
    (128, 2, 3, 17, "star", [20, 3], [2, 1]),
    (128, 5, 50, 2, "chain", [3, 33, 6], [10, 49, 0]),
    (32, 1, 2, 64, "tree", [70], [1]),
]


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2), (SSC, 0), (MEAN, 0), (RESIDUAL, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree(case, delta, dtype, mode, topk):
    d, H, C, T, shape, segs, part = CASES[case]
    gen, rng = seeded(100 * case + 7)
    S = len(segs)
    n_max = max(segs) + 2
    ref = Ref(S, H, d, C, n_max, sum(segs) + 3).fill(segs, part, gen, rng)
    x = tokens(gen, S, H, T, d, dtype)
    if not delta:
        x[4] = x[5] = None
    if mode in (RESIDUAL, MEAN):
        x[3] = None
    count = [T] + [rng.randint(0, T) for _ in range(S - 1)]
    slots = rng.sample(range(S), S)
    cache = on_gpu(ref)
    run_tree(cache, ref, x, draft(rng, S, T, shape), count, slots, mode, topk, dtype)
    same(cache, ref, 1e-6)  # the cache stays as it is


@pytest.mark.parametrize("T", [4, 24])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_indexes_out_of_range(T, dtype):
    """Slots, parents and counts that do not exist, rows to pad with, a slot that comes twice, segments without a page, a table
    entry outside the pool."""
    gen, rng = seeded(3)
    H, d, C = 2, 64, 6
    ref = Ref(6, H, d, C, 9, 40).fill([4, 8, 3, 2, 0, 1], [0, 5, 2, 1, 3, 0], gen, rng)
    ref.table[1][3] = ref.table[1][7] = ref.table[2][0] = -1
    x = tokens(gen, 6, H, T, d, dtype)
    parent = draft(rng, 6, T, "tree")
    parent[0][2], parent[1][1], parent[2][3], parent[2][0] = 2, 99, -5, 0
    cache = on_gpu(ref)
    run_tree(cache, ref, x, parent, [T, T + 9, -3, T, 2, T], [1, 1, 0, -1, 2, 3], GRM, 0, dtype)
    assert ref.status == [INDEX]
    cache.table[3, 1] = 40  # row 3 is slot 3's: not followed, as if it had no page
    ref.table[3][1] = -1
    run_tree(cache, ref, x, draft(rng, 6, T, "tree"), None, [6, -2, 3, 1 << 30, 4, 5], GRM, 0, dtype)
    with pytest.raises(RuntimeError):
        cache.check()
    cache.row[4] = 77  # a row and a position that do not exist: nothing is read or written
    cache.pos[5] = -1
    y = torch.full((6, H, T, d), 7.0, dtype=dtype, device="cuda")
    q, k, v, u, la, be = (gpu(t) for t in x)
    mcl.mc_decode_tree(cache, q, k, v, u, i32(parent), GRM, log_alpha=la, beta=be, slots=i32([4, 5, 4, 5, 4, 5]), y=y)
    assert (y == 7.0).all()
    mcl.mc_tree_accept(cache, k, v, i32(parent), i32([T - 1] * 6), slots=i32([4, 5, 4, 5, 4, 5]))
    assert cache.pos.tolist()[4:] == [3, -1] and cache.status.tolist() == [INDEX]


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SOUP, 0), (SSC, 3), (MEAN, 0), (RESIDUAL, 0)])
@pytest.mark.parametrize("d,C,dtype,delta", [(16, 3, torch.float32, True), (32, 1, torch.bfloat16, False), (64, 4, torch.bfloat16, True),
                                             (128, 5, torch.bfloat16, False), (128, 2, torch.float32, True), (64, 9, torch.float32, False)])
def test_steps(d, C, dtype, delta, mode, topk):
    """Tokens one by one over segment ends, at unlike positions, with rows to pad with."""
    gen, rng = seeded(d + C)
    H, S = 2, 5
    ref = Ref(S, H, d, C, 16, 60).fill([3, 0, 6, 1, 2], [C - 1, 0, 0, C // 2, C - 1], gen, rng)
    cache = on_gpu(ref)
    for t in range(7):
        x = [z[:, :, 0].contiguous() for z in tokens(gen, 4, H, 1, d, dtype)]
        if not delta:
            x[4] = x[5] = None
        if mode in (RESIDUAL, MEAN):
            x[3] = None
        slots = rng.sample([0, 1, 2, 3, 4, -1], 4)
        y = torch.full((4, H, d), 7.0, dtype=dtype, device="cuda")
        q, k, v, u, la, be = (gpu(z) for z in x)
        mcl.mc_decode_step_paged(cache, q, k, v, u, mode, topk, log_alpha=la, beta=be, slots=i32(slots), y=y)
        want = ref.step(*x, slots, mode, topk)
        for b in range(4):
            if b in want:
                near(y[b], want[b], TOL[dtype])
            else:
                assert (y[b] == 7.0).all()
    same(cache, ref)


def test_a_slot_named_twice_and_an_empty_pool_and_a_full_table():
    gen, rng = seeded(11)
    H, d, C = 1, 16, 2
    ref = Ref(4, H, d, C, 3, 7).fill([2, 2, 1, 0], [1, 1, 1, 1], gen, rng)  # two free pages
    cache = on_gpu(ref)
    x = [z[:, :, 0].contiguous() for z in tokens(gen, 4, H, 1, d, torch.float32)]
    q, k, v, u, la, be = (gpu(z) for z in x)
    def step(slots):
        y = torch.full((len(slots), H, d), 7.0, device="cuda")
        n = len(slots)
        mcl.mc_decode_step_paged(cache, q[:n], k[:n], v[:n], u[:n], GRM, slots=i32(slots), y=y)
        want = ref.step(x[0][:n], x[1][:n], x[2][:n], x[3][:n], None, None, slots, GRM, 0)
        for b in range(n):
            assert torch.allclose(y[b].double().cpu(), want[b], atol=1e-4) if b in want else bool((y[b] == 7.0).all())
        same(cache, ref)
    step([1, 0, 1, 9])  # slot 1's second row is not run; both others complete a segment: the pool is empty then
    assert ref.status == [INDEX] and sum(r == 0 for r in ref.refs) == 0
    step([2, 3])  # no page for either
    assert ref.status == [INDEX | NONE_FREE]
    for _ in range(3):
        step([2, 0, 3, 1])  # past the table's end, too
    assert ref.status == [INDEX | NONE_FREE | TABLE_FULL]
    for _ in range(3):
        step([3, 1])


@pytest.mark.parametrize("d,C,T,dtype,delta", [(16, 3, 7, torch.float32, True), (32, 1, 64, torch.bfloat16, True),
                                               (64, 6, 33, torch.bfloat16, False), (128, 40, 64, torch.bfloat16, True),
                                               (128, 7, 12, torch.float32, False), (64, 2, 1, torch.float32, True)])
def test_accept(d, C, T, dtype, delta):
    gen, rng = seeded(d + T)
    H, S = 3, 5
    n_max = 5 + T // C + 1
    ref = Ref(S, H, d, C, n_max, S * n_max).fill([3, 0, 4, 1, 2], [C - 1, 0, 0, C // 2, 1 % C], gen, rng)
    cache = on_gpu(ref)
    for turn in range(2):
        x = tokens(gen, S, H, T, d, dtype)
        if not delta:
            x[4] = x[5] = None
        parent = draft(rng, S, T, "chain" if turn else "tree")
        last = [T - 1, -1, T // 2, T + 5, T - 1]
        slots = [2, 1, 0, 3, 4] if turn else [4, 2, -1, 0, 2]
        mcl.mc_tree_accept(cache, gpu(x[1]), gpu(x[2]), i32(parent), i32(last), log_alpha=gpu(x[4]), beta=gpu(x[5]), slots=i32(slots))
        ref.accept(x[1], x[2], x[4], x[5], parent, last, slots)
        same(cache, ref)
        assert ref.status == [INDEX]


def test_accept_on_an_empty_pool():
    gen, rng = seeded(2)
    ref = Ref(3, 2, 16, 2, 4, 6).fill([1, 2, 0], [1, 0, 1], gen, rng)  # three free pages for eleven segments
    cache = on_gpu(ref)
    x = tokens(gen, 3, 2, 9, 16, torch.float32)
    parent = draft(rng, 3, 9, "chain")
    mcl.mc_tree_accept(cache, gpu(x[1]), gpu(x[2]), i32(parent), i32([8, 6, 7]))
    ref.accept(x[1], x[2], None, None, parent, [8, 6, 7], None)
    same(cache, ref)
    assert ref.status == [NONE_FREE | TABLE_FULL]


@pytest.mark.parametrize("S", [1, 5, 33])
def test_forks(S):
    """Swaps, cycles, samples, freed slots, numbers out of range, again and again."""
    gen, rng = seeded(S)
    H, d, C, n_max = 2, 32, 4, 5
    segs = [rng.randrange(n_max + 1) for _ in range(S)]
    ref = Ref(S, H, d, C, n_max, sum(segs) + 2)
    rng.shuffle(ref.row)
    ref.fill(segs, [rng.randrange(C) for _ in segs], gen, rng)
    cache = on_gpu(ref)
    todo = [list(range(S)), list(range(1, S)) + [0], [0] * S, [rng.randrange(S) for _ in range(S)],
            [rng.randrange(-3, S + 2) for _ in range(S)], [x if x % 3 else -1 for x in range(S)], [-1] * S]
    for src in todo[:3] + todo[3:5] + [todo[1]] + todo[5:]:
        mcl.mc_pages_fork(cache, i32(src))
        ref.fork(src)
        same(cache, ref, 1e-7)
    assert sum(ref.refs) == 0


@pytest.mark.parametrize("room", [-3, 0, 5])
def test_compact(room):
    gen, rng = seeded(room + 50)
    H, d, C = 3, 64, 4
    ref = Ref(6, H, d, C, 5, 1100)
    rng.shuffle(ref.row)
    ref.fill([3, 5, 0, 2, 1, 4], [1, 0, 3, 2, 0, 1], gen, rng)
    ref.fork([0, 1, -1, 0, 0, 5])
    live = sum(r > 0 for r in ref.refs)
    src = on_gpu(ref)
    into = mcl.PagedCache(8, H, d, C, 7, live + room)
    for t in (into.refs, into.pos, into.row, into.table):
        t.fill_(3)  # what it held is gone
    before = {n: getattr(src, n).clone() for n in FLOATS + INTS}
    mcl.mc_pages_compact(into, src)
    to = ref.compact(8, 7, live + room)
    for n in INTS:
        assert getattr(into, n).cpu().tolist() == getattr(to, n), n
    for n in ("pages", "kbar"):
        m = min(live, live + room)
        assert torch.equal(getattr(into, n)[:m].double().cpu(), getattr(to, n)[:m]), n
    assert torch.equal(into.online[:6].double().cpu(), to.online[:6]) and torch.equal(into.ksum[:6].double().cpu(), to.ksum[:6])
    assert all(torch.equal(getattr(src, n), x) for n, x in before.items())
    assert to.status == [NONE_FREE if room < 0 else 0]


@pytest.mark.parametrize("d,C,L,dtype", [(16, 5, 23, torch.float32), (64, 16, 64, torch.bfloat16), (128, 33, 200, torch.bfloat16), (32, 50, 20, torch.float32)])
def test_load(d, C, L, dtype):
    gen, rng = seeded(L)
    H = 2
    n_max = L // C + 1
    ref = Ref(3, H, d, C, n_max, 3 * n_max)
    rng.shuffle(ref.row)
    ref.fill([1, n_max, 0], [0, 1, 0], gen, rng)
    cache = on_gpu(ref)
    k = torch.randn(H, L, d, generator=gen).to(dtype)
    states = torch.randn(H, -(-L // C), d, d, generator=gen)
    for slot in (1, 2, 1):
        mcl.mc_pages_load(cache, slot, k.cuda(), states.cuda())
        ref.load(slot, k, states)
        same(cache, ref, 1e-6)


def test_load_without_enough_pages():
    gen, rng = seeded(9)
    ref = Ref(2, 1, 16, 2, 4, 5).fill([0, 3], [0, 0], gen, rng)
    cache = on_gpu(ref)
    k, states = torch.randn(1, 7, 16, generator=gen), torch.randn(1, 4, 16, 16, generator=gen)
    mcl.mc_pages_load(cache, 0, k.cuda(), states.cuda())
    ref.load(0, k, states)
    same(cache, ref, 1e-6)
    assert ref.status == [NONE_FREE]


@pytest.mark.parametrize("T", [6, 20])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 1)])
def test_nan_where_nothing_is_read(mode, topk, delta, T):
    """NaN in free pages, in a begun segment's memory that nothing has entered, in nodes that are no ancestors or beyond the
    count, in other heads, in rows to pad with, and in segments that SSC leaves out."""
    gen, rng = seeded(21)
    H, d, C, nan = 2, 64, 8, float("nan")
    ref = Ref(3, H, d, C, 6, 14).fill([5, 3, 2], [0, 4, 5], gen, rng)
    x = tokens(gen, 3, H, T, d, torch.bfloat16)
    if not delta:
        x[4] = x[5] = None
    parent = [[-1] * T for _ in range(3)]
    parent[1] = draft(rng, 1, T, "chain")[0]
    slots, count = [0, 1, -1], [T, T - 2, T]
    want = ref.tree(*x, parent, count, slots, mode, topk)
    cache = on_gpu(ref)
    free = [p for p in range(14) if ref.refs[p] == 0]
    cache.pages[free], cache.kbar[free] = nan, nan
    cache.online[ref.row[0]], cache.ksum[ref.row[0]] = nan, nan
    x = [gpu(t) for t in x]
    for t in x:
        if t is not None:
            t[0, :, 3], t[1, :, T - 2:], t[2] = nan, nan, nan
    if mode == SSC:  # slot 0: a segment whose scores are far below the others'
        r, far = ref.row[0], cache.table[ref.row[0], 1].item()
        cache.kbar[far], ref.kbar[far] = 0, 0
        x[3][0, :, [j for j in range(T) if j != 3]] = 4.0
        u = x[3].cpu()
        for i in (0, 2, 3, 4):
            ref.kbar[ref.table[r][i]] = ref.kbar[ref.table[r][i]].abs()
            cache.kbar[ref.table[r][i]] = cache.kbar[ref.table[r][i]].abs()
        u[0, :, 3] = 0
        u[1, :, T - 2:] = 0
        ok = [torch.nan_to_num(t.cpu()) if t is not None else None for t in x]
        want = ref.tree(*ok[:3], u, *ok[4:], parent, count, slots, mode, topk)
        cache.pages[far] = nan
    y = torch.full((3, H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    mcl.mc_decode_tree(cache, x[0], x[1], x[2], x[3], i32(parent), mode, topk, log_alpha=x[4], beta=x[5], count=i32(count),
                       slots=i32(slots), y=y)
    y = y.double().cpu()
    assert (y[2] == 7).all() and (y[1, :, T - 2:] == 7).all() and torch.isnan(y[0, :, 3]).all()
    for (b, j), z in want.items():
        if (b, j) != (0, 3):
            near(y[b, :, j], z, 1.5e-2)  # of one node's largest value


def test_equal_scores_go_to_the_older_segment():
    gen, rng = seeded(8)
    ref = Ref(1, 1, 32, 4, 8, 9).fill([7], [1], gen, rng)
    ref.kbar[:] = ref.kbar[:1]
    cache = on_gpu(ref)
    x = tokens(gen, 1, 1, 3, 32, torch.float32)
    for topk in (0, 1, 3, 6, 7, 8, 1 << 30):
        run_tree(cache, ref, x, [[-1, 0, 0]], None, None, SSC, topk, torch.float32)


@pytest.mark.parametrize("delta", [False, True])
def test_a_server(delta):
    """Prefill, load, fork, drafts read and accepted, steps, frees and a compaction: every token's output is that of a dense
    64-bit cache, and of mc_decode_step token by token."""
    H, d, C, L = 2, 64, 16, 40
    gen, rng = seeded(17)
    x = tokens(gen, 1, H, L, d, torch.bfloat16)
    q, k, v, u, la, be = (gpu(t) for t in x)
    if delta:
        _, states = mcl.mc_forward_delta(q, k, v, u, la, be, C, GRM)
    else:
        _, states = mcl.mc_forward(q, k, v, u, C, GRM)
        x[4] = x[5] = None
    cache, ref = mcl.PagedCache(4, H, d, C, 8, 20), Ref(4, H, d, C, 8, 20)
    mcl.mc_pages_load(cache, 2, k[0], states[0])
    ref.load(2, x[1][0], states[0].cpu())
    mcl.mc_pages_fork(cache, i32([2, 2, 2, -1]))
    ref.fork([2, 2, 2, -1])
    dense = mcl.DecodeCache(1, H, d, C, 8)
    dense.states[0, :, :2], dense.kbar[0, :, :2] = states[0, :, :2], torch.stack([k[0, :, i * C:(i + 1) * C].float().mean(1) for i in range(2)], 1)
    dense.online[0], dense.ksum[0], dense.t = states[0, :, 2], k[0, :, 32:].float().sum(1), L
    for turn in range(4):
        T = 12
        x = tokens(gen, 3, H, T, d, torch.bfloat16)
        if not delta:
            x[4] = x[5] = None
        parent = draft(rng, 3, T, "chain" if turn % 2 else "tree")
        slots, last = [1, 0, 2], [T - 1, 5, -1]
        y = run_tree(cache, ref, x, parent, None, slots, GRM, 0, torch.bfloat16)
        path, j = [], T - 1
        while j >= 0:
            path.insert(0, j)
            j = parent[0][j]
        for j in path:  # slot 1 goes on along the path to its last node
            tok = [gpu(t[:1, :, j].contiguous()) if t is not None else None for t in x]
            z = mcl.mc_decode_step_delta(dense, *tok, GRM) if delta else mcl.mc_decode_step(dense, *tok[:4], GRM)
            near(y[0, :, j].float(), z[0].double().cpu(), 2e-2)
        mcl.mc_tree_accept(cache, gpu(x[1]), gpu(x[2]), i32(parent), i32(last), log_alpha=gpu(x[4]), beta=gpu(x[5]), slots=i32(slots))
        ref.accept(x[1], x[2], x[4], x[5], parent, last, slots)
        same(cache, ref)
        tok = [t[:, :, 0].contiguous() if t is not None else None for t in tokens(gen, 2, H, 1, d, torch.bfloat16)]
        if not delta:
            tok[4] = tok[5] = None
        got = mcl.mc_decode_step_paged(cache, *(gpu(t) for t in tok[:4]), GRM, log_alpha=gpu(tok[4]), beta=gpu(tok[5]), slots=i32([0, 2]))
        want = ref.step(*tok, [0, 2], GRM, 0)
        near(got.float(), torch.stack([want[0], want[1]]), 1e-2)
    mcl.mc_pages_fork(cache, i32([0, 1, -1, 1]))
    ref.fork([0, 1, -1, 1])
    same(cache, ref)
    live = sum(r > 0 for r in ref.refs)
    small = mcl.PagedCache(4, H, d, C, 8, live)
    mcl.mc_pages_compact(small, cache)
    same(small, ref.compact(4, 8, live))
    x = tokens(gen, 4, H, 9, d, torch.bfloat16)
    if not delta:
        x[4] = x[5] = None
    run_tree(small, ref.compact(4, 8, live), x, draft(rng, 4, 9, "tree"), None, None, GRM, 0, torch.bfloat16)
    small.check()


def pair(T, dtype=torch.bfloat16):
    gen, rng = seeded(T)
    ref = Ref(3, 2, 64, 8, 12, 40).fill([9, 4, 6], [7, 0, 3], gen, rng)
    x = tokens(gen, 3, 2, T, 64, dtype)
    return ref, [gpu(t) for t in x], i32(draft(rng, 3, T, "tree"))


@pytest.mark.parametrize("T", [5, 30])
def test_graphs_and_streams(T):
    """A captured tree and step, replayed as positions move on; the same on side streams at once; runs repeat bit for bit."""
    ref, x, parent = pair(T)
    a, b = on_gpu(ref), on_gpu(ref)
    tree = lambda c: mcl.mc_decode_tree(c, *x[:4], parent, GRM, log_alpha=x[4], beta=x[5])  # noqa: E731
    tok = [t[:, :, 0].contiguous() for t in x]
    step = lambda c: mcl.mc_decode_step_paged(c, *tok[:4], GRM, log_alpha=tok[4], beta=tok[5])  # noqa: E731
    want = []
    for _ in range(4):
        want.append((tree(a), step(a)))
    warm = on_gpu(ref)
    tree(warm), step(warm)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yt = tree(b)
    with torch.cuda.graph(g2):
        ys = step(b)
    for wt, ws in want:
        g.replay()
        g2.replay()
        assert torch.equal(yt, wt) and torch.equal(ys, ws)
    for n in FLOATS + INTS:
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert a.status.item() == 0
    c = on_gpu(ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(5):
        for s in streams:  # several reads of one cache at once
            with torch.cuda.stream(s):
                outs.append(tree(c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0][0]) for o in outs)


def test_views_and_parts_of_a_batch():
    """Index arrays and gates that begin at any element, and a batch smaller than the cache."""
    ref, x, parent = pair(6, torch.float32)
    cache = on_gpu(ref)
    whole = mcl.mc_decode_tree(cache, *x[:4], parent, GRM, log_alpha=x[4], beta=x[5])
    for b in range(3):
        part = [t[b:b + 1] for t in x]
        slots = torch.tensor([9, b], dtype=torch.int32, device="cuda")[1:]
        got = mcl.mc_decode_tree(cache, *part[:4], parent[b:b + 1], GRM, log_alpha=part[4], beta=part[5], slots=slots)
        assert torch.allclose(got[0], whole[b], rtol=1e-5, atol=1e-5)
    bad = x[0].transpose(2, 3).contiguous().transpose(2, 3)
    with pytest.raises(ValueError):
        mcl.mc_decode_tree(cache, bad, *x[1:4], parent, GRM)
    with pytest.raises(TypeError):
        mcl.mc_decode_tree(cache, *x[:4], parent.long(), GRM)
    with pytest.raises(TypeError):
        mcl.mc_decode_tree(cache, x[0].half(), *x[1:4], parent, GRM)
    with pytest.raises(ValueError):
        mcl.mc_decode_tree(cache, *(t[:, :1].contiguous() for t in x[:4]), parent, GRM)
    with pytest.raises(mcl.MCError):
        mcl.mc_decode_tree(cache, *x[:3], None, parent, GRM)
    with pytest.raises(mcl.MCError):
        mcl.mc_decode_tree(cache, *x[:4], parent, GRM, log_alpha=x[4])


@pytest.mark.parametrize("T", [3, 12])
def test_more_pages_than_32_bits_reach(T):
    """Pages beyond 2^31 floats."""
    H, d = 16, 128
    P = (1 << 31) // (H * d * d) + 3
    gen, rng = seeded(1)
    small = Ref(1, H, d, 4, 4, 3).fill([2], [1], gen, rng)
    cache = mcl.PagedCache(1, H, d, 4, 4, P)
    for n in ("online", "ksum", "pos"):
        getattr(cache, n).copy_(torch.as_tensor(getattr(small, n)))
    for i in range(2):
        p = P - 1 - i
        cache.pages[p], cache.kbar[p] = small.pages[small.table[0][i]].float().cuda(), small.kbar[small.table[0][i]].float().cuda()
        cache.table[0, i] = p
    cache.refs[:] = 1
    cache.refs[P - 3] = 0  # the only free page: that of the segment completed below
    x = tokens(gen, 1, H, T, d, torch.bfloat16)
    parent = draft(rng, 1, T, "chain")
    run_tree(cache, small, x, parent, None, None, GRM, 0, torch.bfloat16)
    mcl.mc_tree_accept(cache, gpu(x[1]), gpu(x[2]), i32(parent), i32([2]))
    small.accept(x[1], x[2], None, None, parent, [2], None)
    near(cache.pages[P - 3].double().cpu(), small.pages[small.table[0][2]], 1e-4)
    assert cache.table[0, 2].item() == P - 3 and cache.status.item() == 0
    del cache
    torch.cuda.empty_cache()


def test_many_sequences():
    """A full batch: 1024 sequences of a small model, more than a plan's threads can scan pages for in one turn."""
    S, H, d, C = 1024, 1, 16, 2
    gen, rng = seeded(4)
    segs = [rng.randrange(3) for _ in range(S)]
    ref = Ref(S, H, d, C, 4, sum(segs) + S + 5).fill(segs, [1] * S, gen, rng)
    cache = on_gpu(ref)
    x = [z[:, :, 0].contiguous() for z in tokens(gen, S, H, 1, d, torch.float32)]
    got = mcl.mc_decode_step_paged(cache, *(gpu(z) for z in x[:4]), GRM)
    want = ref.step(*x[:4], None, None, None, GRM, 0)
    near(got, torch.stack([want[b] for b in range(S)]), 1e-4)
    same(cache, ref)
    src = [rng.randrange(-1, S) for _ in range(S)]
    mcl.mc_pages_fork(cache, i32(src))
    ref.fork(src)
    same(cache, ref)


# n_max so large that a draft of few nodes takes more than one launch (the capacity says so, not what is cached): every kernel
# for 1, 2, 4 and 8 nodes
@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2), (SOUP, 0), (MEAN, 0), (RESIDUAL, 0)])
@pytest.mark.parametrize("T", [1, 2, 3, 8])
@pytest.mark.parametrize("d,H,n_max,dtype", [(16, 44, 1000, torch.float32), (32, 22, 512, torch.bfloat16), (64, 12, 250, torch.bfloat16),
                                             (128, 8, 90, torch.float32), (128, 7, 100, torch.bfloat16)])
def test_few_nodes_over_much_room(d, H, n_max, dtype, T, mode, topk):
    gen, rng = seeded(d + T)
    ref = Ref(2, H, d, 3, n_max, 16).fill([9, 4], [1, 0], gen, rng)
    x = tokens(gen, 2, H, T, d, dtype)
    if (T + mode) % 2:
        x[4] = x[5] = None
    cache = on_gpu(ref)
    run_tree(cache, ref, x, draft(rng, 2, T, "tree"), [T, max(T - 1, 1)], [1, 0], mode, topk, dtype)


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_read_nothing_else(dtype, mode, topk):
    """A step with NaN in free pages, in rows to pad with, in begun segments that nothing has entered; a segment without a page and
    one whose page does not exist; inputs that are parts of larger tensors."""
    gen, rng = seeded(31)
    H, d, C, nan = 2, 64, 4, float("nan")
    ref = Ref(4, H, d, C, 8, 24).fill([5, 3, 2, 4], [0, 3, 1, 3], gen, rng)
    ref.table[1][0] = ref.table[3][2] = -1
    x = [z[:, :, 0].contiguous() for z in tokens(gen, 4, H, 1, d, dtype)]
    cache = on_gpu(ref)
    cache.table[1, 0] = 24  # past the pool: not followed
    free = [p for p in range(24) if ref.refs[p] == 0]
    cache.pages[free], cache.kbar[free] = nan, nan
    cache.online[0], cache.ksum[0] = nan, nan
    wide = [torch.full((6, *z.shape[1:]), nan, dtype=dtype, device="cuda") for z in x]
    for w, z in zip(wide, x):
        w[1:4] = z[:3].cuda()
    part = [w[1:5] for w in wide]  # the fourth row is NaN and nobody's
    y = torch.full((4, H, d), 7.0, dtype=dtype, device="cuda")
    slots = torch.tensor([9, 3, 0, 1, -1], dtype=torch.int32, device="cuda")[1:]
    mcl.mc_decode_step_paged(cache, *part[:4], mode, topk, log_alpha=part[4], beta=part[5], slots=slots, y=y)
    want = ref.step(*x, [3, 0, 1, -1], mode, topk)
    for b in range(3):
        near(y[b], want[b], TOL[dtype])
    assert (y[3] == 7).all() and cache.pos.tolist() == ref.pos and cache.refs.tolist() == ref.refs
    for b, i in ((3, 4), (1, 3)):  # the segments that the call completed
        p = cache.table[b, i].item()
        assert p == ref.table[b][i]
        near(cache.pages[p].double().cpu(), ref.pages[p], 1e-4)
        near(cache.kbar[p].double().cpu(), ref.kbar[p], 1e-4)


def test_steps_beside_other_work():
    """Small steps while another stream keeps the GPU busy, so that CTAs of one call come up at unlike times; every token completes
    a segment, which changes how many of them have work."""
    gen, rng = seeded(13)
    H, d, C = 2, 32, 1
    ref = Ref(3, H, d, C, 40, 130).fill([0, 2, 1], [0, 0, 0], gen, rng)
    cache = on_gpu(ref)
    xs = [[z[:, :, 0].contiguous() for z in tokens(gen, 3, H, 1, d, torch.float32)] for _ in range(30)]
    on = [[gpu(z) for z in x] for x in xs]
    side = torch.cuda.Stream()
    m = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            m = torch.relu(m + 1.0) * 0.5
            m = (m @ m) * 1e-5
    ys = [mcl.mc_decode_step_paged(cache, *x[:4], GRM, log_alpha=x[4], beta=x[5]) for x in on]
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        want = ref.step(*x, None, GRM, 0)
        near(y, torch.stack([want[b] for b in range(3)]), 1e-4)
    same(cache, ref)


def test_a_given_stream_and_two_graphs():
    """Calls on a stream given by name, and graphs of two caches replayed at once: neither touches the other's work."""
    ref, x, parent = pair(5)
    tok = [t[:, :, 0].contiguous() for t in x]
    a, b, c = on_gpu(ref), on_gpu(ref), on_gpu(ref)
    last = i32([4, 3, 2])
    everything = lambda k, **s: (  # noqa: E731
        mcl.mc_decode_tree(k, *x[:4], parent, GRM, log_alpha=x[4], beta=x[5], **s),
        mcl.mc_tree_accept(k, x[1], x[2], parent, last, log_alpha=x[4], beta=x[5], **s),
        mcl.mc_decode_step_paged(k, *tok[:4], GRM, log_alpha=tok[4], beta=tok[5], **s),
        mcl.mc_pages_fork(k, src, **s))
    src = i32([1, 2, 0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [everything(a) for _ in range(3)]
    torch.cuda.synchronize()
    got = [everything(c, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[2], g[2])
    same_bits = lambda p, q: all(torch.equal(getattr(p, n), getattr(q, n)) for n in FLOATS + INTS)  # noqa: E731
    assert same_bits(a, c) and a.status.item() == 0
    d = on_gpu(ref)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in (b, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t = mcl.mc_decode_tree(k, *x[:4], parent, GRM, log_alpha=x[4], beta=x[5])
            mcl.mc_tree_accept(k, x[1], x[2], parent, last, log_alpha=x[4], beta=x[5])
            z = mcl.mc_decode_step_paged(k, *tok[:4], GRM, log_alpha=tok[4], beta=tok[5])
            mcl.mc_pages_fork(k, src)
        graphs.append(g)
        outs.append((t, z))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for w in want:
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t, z in outs:
            assert torch.equal(t, w[0]) and torch.equal(z, w[2])
    assert same_bits(a, b) and same_bits(a, d)


def test_tokens_that_are_missing_are_refused():
    ref, x, parent = pair(4)
    cache = on_gpu(ref)
    tok = [t[:, :, 0].contiguous() for t in x]
    for i in range(1, 3):
        with pytest.raises(TypeError):
            mcl.mc_decode_tree(cache, *(None if i == j else t for j, t in enumerate(x[:4])), parent, GRM)
        with pytest.raises(TypeError):
            mcl.mc_decode_step_paged(cache, *(None if i == j else t for j, t in enumerate(tok[:4])), GRM)
    with pytest.raises(TypeError):
        mcl.mc_tree_accept(cache, x[1], None, parent, i32([0, 0, 0]))
    for call in (lambda: mcl.mc_tree_accept(cache, x[1], x[2], parent, None), lambda: mcl.mc_tree_accept(cache, x[1], x[2], None, i32([0, 0, 0])),
                 lambda: mcl.mc_decode_tree(cache, *x[:4], None, GRM)):
        with pytest.raises(mcl.MCError):
            call()
    same(cache, ref, 1e-7)
