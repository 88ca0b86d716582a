"""Calls of the paged cache that the other tests' sizes do not reach.  Tolerances as in test_paged_gpu.py: of an output's largest
value 1e-4 with fp32 inputs, 1e-2 with bf16 ones; what is copied or counted is equal."""
import copy

import pytest
import torch

import memory_caching_linear_gb300 as mcl
from paged_ref import GRM, MEAN, RESIDUAL, SSC, TABLE_FULL, Ref, draft, seeded, tokens
from test_paged_gpu import gpu, i32, near, on_gpu, run_tree, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [(1 << 31) - 1, (1 << 31) - 20, 1 << 30])
@pytest.mark.parametrize("d,L,dtype", [(16, 2, torch.float32), (64, 37, torch.bfloat16), (128, 1000, torch.bfloat16)])
def test_a_prompt_in_a_segment_that_never_ends(d, L, dtype, C):
    """L + seg_len - 1 past 32 bits: every head has its own memory and key sum, and steps and drafts go on from them."""
    gen, rng = seeded(d)
    H, T = 3, 9
    ref = Ref(2, H, d, C, 2, 3)
    cache = on_gpu(ref)
    k = torch.randn(H, L, d, generator=gen).to(dtype)
    states = torch.randn(H, 1, d, d, generator=gen)
    mcl.mc_pages_load(cache, 1, k.cuda(), states.cuda())
    ref.load(1, k, states)
    assert torch.equal(cache.online[1].cpu(), states[:, 0])
    same(cache, ref, 1e-6)
    x = tokens(gen, 1, H, T, d, dtype)
    run_tree(cache, ref, x, draft(rng, 1, T, "tree"), None, [1], GRM, 0, dtype)
    one = [t[:, :, 0].contiguous() for t in x]
    y = mcl.mc_decode_step_paged(cache, *(gpu(t) for t in one[:4]), GRM, log_alpha=gpu(one[4]), beta=gpu(one[5]), slots=i32([1]))
    near(y, ref.step(*one, [1], GRM, 0)[0], 1e-4 if dtype == torch.float32 else 1e-2)
    same(cache, ref)


@pytest.mark.parametrize("delta", [False, True])
def test_rows_to_pad_with_are_not_read_by_an_acceptance(delta):
    """Nodes and parents that do not exist, in rows of nobody: nothing is reported, nothing changes but the other rows'."""
    gen, rng = seeded(40)
    H, d, C, T = 2, 64, 5, 12
    ref = Ref(4, H, d, C, 8, 30).fill([2, 1, 0, 3], [4, 0, 3, 2], gen, rng)
    cache = on_gpu(ref)
    x = tokens(gen, 4, H, T, d, torch.bfloat16)
    if not delta:
        x[4] = x[5] = None
    parent, last, slots = draft(rng, 4, T, "tree"), [T - 1, 5, 7, 3], [3, -1, 0, -1]
    garbage = [1 << 30, -(1 << 31), 77, -2] * (T // 4)
    on = [gpu(t) for t in x]
    for t in on[1:3] + on[4:]:
        if t is not None:
            t[1], t[3] = float("nan"), float("nan")
    for junk in ([T, 1 << 30], [-9, T - 1]):
        mcl.mc_tree_accept(cache, on[1], on[2], i32([parent[0], garbage, parent[2], garbage]), i32([last[0], junk[0], last[2], junk[1]]),
                           log_alpha=on[4], beta=on[5], slots=i32(slots))
        ref.accept(x[1], x[2], x[4], x[5], parent, last, slots)
        assert ref.status == [0] and cache.status.tolist() == [0]
        same(cache, ref)
    cache.check()


@pytest.mark.parametrize("T,d,dtype", [(7, 64, torch.bfloat16), (20, 64, torch.bfloat16), (20, 32, torch.float32), (12, 128, torch.float32)])
@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2), (MEAN, 0)])
def test_drafts_where_the_table_ends(T, d, dtype, mode, topk):
    """Whether a path's segments would find a place does not matter to what is read: the same as with a table of room; the
    acceptance loses them and says so."""
    gen, rng = seeded(T + d)
    H, C, S = 2, 2, 2
    ref = Ref(S, H, d, C, 4, 12).fill([3, 4], [1, 0], gen, rng)
    wide = mcl.PagedCache(S, H, d, C, 40, 12)
    cache = on_gpu(ref)
    for n in ("pages", "kbar", "online", "ksum", "refs", "pos", "row"):
        getattr(wide, n).copy_(getattr(cache, n))
    wide.table[:, :4] = cache.table
    x = tokens(gen, S, H, T, d, dtype)
    if mode == MEAN:
        x[3] = None
    parent = draft(rng, S, T, "chain")
    y = run_tree(cache, ref, x, parent, None, None, mode, topk, dtype)
    on = [gpu(t) for t in x]
    z = mcl.mc_decode_tree(wide, *on[:4], i32(parent), mode, topk, log_alpha=on[4], beta=on[5])
    near(z, y.double().cpu(), 1e-4 if dtype == torch.float32 else 1e-2)
    assert cache.status.item() == 0 and wide.status.item() == 0
    mcl.mc_tree_accept(cache, on[1], on[2], i32(parent), i32([T - 1, 0]), log_alpha=on[4], beta=on[5])
    ref.accept(x[1], x[2], x[4], x[5], parent, [T - 1, 0], None)
    assert ref.status == [TABLE_FULL]
    same(cache, ref)


def test_a_copied_cache_goes_its_own_way():
    gen, rng = seeded(12)
    H, d, C, T = 2, 64, 4, 6
    ref = Ref(2, H, d, C, 8, 20).fill([3, 2], [3, 1], gen, rng)
    cache = on_gpu(ref)
    x = [z[:, :, 0].contiguous() for z in tokens(gen, 2, H, 1, d, torch.float32)]
    on = [gpu(z) for z in x]
    step = lambda c: mcl.mc_decode_step_paged(c, *on[:4], GRM, log_alpha=on[4], beta=on[5])  # noqa: E731
    step(cache)
    ref.step(*x, None, GRM, 0)
    twin, ref2 = copy.deepcopy(cache), copy.deepcopy(ref)
    for _ in range(2):
        y, want = step(twin), ref2.step(*x, None, GRM, 0)
        near(y, torch.stack([want[0], want[1]]), 1e-4)
    same(twin, ref2)
    same(cache, ref)  # as it was when it was copied


def test_check_waits_for_every_stream():
    """A bad index in a call on a stream that is busy when check() is called on another."""
    gen, rng = seeded(14)
    ref = Ref(2, 1, 16, 4, 4, 8).fill([1, 1], [0, 0], gen, rng)
    cache = on_gpu(ref)
    on = [gpu(z[:, :, 0].contiguous()) for z in tokens(gen, 2, 1, 1, 16, torch.float32)]
    side, m = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    slots = i32([0, 5])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            m = (m @ m) * 1e-5
        mcl.mc_decode_step_paged(cache, *on[:4], GRM, slots=slots)
    with pytest.raises(RuntimeError, match="index"):
        cache.check()
    cache.check()
    assert cache.status.item() == 0


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (32, torch.bfloat16), (64, torch.float32)])
@pytest.mark.parametrize("mode,topk", [(GRM, 0), (MEAN, 0), (RESIDUAL, 0), (SSC, 3)])
@pytest.mark.parametrize("T", [5, 21])
def test_segments_without_a_page(T, mode, topk, d, dtype):
    """Segments that found none -- first, last, every other, all of a sequence -- under every aggregation; NaN in free pages."""
    gen, rng = seeded(d + T)
    H, C, S = 3, 4, 4
    ref = Ref(S, H, d, C, 12, 40).fill([7, 5, 9, 4], [1, 0, 3, 2], gen, rng)
    gone = {0: [0], 1: [4], 2: [0, 2, 4, 6, 8], 3: [0, 1, 2, 3]}
    for b, which in gone.items():
        for i in which:
            ref.refs[ref.table[b][i]] = 0
            ref.table[b][i] = -1
    cache = on_gpu(ref)
    free = [p for p in range(40) if ref.refs[p] == 0]
    cache.pages[free], cache.kbar[free] = float("nan"), float("nan")
    x = tokens(gen, S, H, T, d, dtype)
    if mode in (MEAN, RESIDUAL):
        x[3] = None
    run_tree(cache, ref, x, draft(rng, S, T, "tree"), [T, T - 1, T, T], [2, 0, 3, 1], mode, topk, dtype)
    one = [None if t is None else t[:, :, 0].contiguous() for t in x]
    on = [gpu(t) for t in one]
    y = mcl.mc_decode_step_paged(cache, *on[:4], mode, topk, log_alpha=on[4], beta=on[5])
    want = ref.step(*one, None, mode, topk)
    near(y, torch.stack([want[b] for b in range(S)]), 1e-4 if dtype == torch.float32 else 1e-2)
