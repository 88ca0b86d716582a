"""The paged step and the drafts where every CTA has many memories: ring and operand slots used again and again, sums over a
head's memories, several heads after one another, ranges cut across heads and sequences.

16 heads against the 64-bit form on three of them (each in another part of the line of memories).  Tolerances, of an output's
largest value: 1e-4 with fp32 inputs, 1e-2 with bf16 ones; what is counted is equal.  For the sparse router the cached mean keys and
the router's inputs are multiples of 1/8 below 4: their products and sums are exact in 32 bits, equal ones among them."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from paged_ref import FLOATS, GRM, INTS, MEAN, RESIDUAL, SSC, Ref, draft, seeded, tokens
from test_paged_gpu import TOL, gpu, i32, near

pytestmark = pytest.mark.gpu
H, HEADS = 16, [0, 7, 15]
LONG = [40, 33, 41, 0, 37, 12, 39, 40]                     # 242 segments: 26 memories a CTA and more
SHORT = [3, 1, 4, 2, 5, 0, 2, 6, 1, 1, 3, 5, 2, 2, 4, 1, 6, 3, 0, 2, 5, 4, 1, 2]  # 65: seven, of several heads
SHAPES = {"long": LONG, "short": SHORT}


def sampled(d, C, segs, seed, exact_scores):
    """A cache of 16 heads and its 64-bit form on three."""
    gen, rng = seeded(seed)
    S, n_max = len(segs), max(segs) + 3
    ref = Ref(S, len(HEADS), d, C, n_max, sum(segs) + 2 * S)
    rng.shuffle(ref.row)
    part = [C - 1 if x % 3 == 0 else 0 if x % 3 == 1 else C // 2 for x in range(S)]
    ref.fill(segs, part, gen, rng)
    cache = mcl.PagedCache(S, H, d, C, n_max, ref.P)
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda t: torch.randn(t.shape, device="cuda", generator=g)  # noqa: E731
    for name, size in (("pages", 0.5), ("kbar", 0.5), ("online", 0.3), ("ksum", 0.3)):
        t = getattr(cache, name)
        t.copy_(rnd(t) * size)
        if name == "kbar" and exact_scores:
            t.copy_(((t * 8).round() / 8).clamp(-3, 3))
        getattr(ref, name).copy_(t[:, HEADS])
    for name in INTS:
        getattr(cache, name).copy_(torch.tensor(getattr(ref, name)))
    return cache, ref, gen, rng


def inputs(gen, B, T, d, dtype, delta, mode):
    x = tokens(gen, B, H, T, d, dtype)
    if mode == SSC:
        x[3] = ((x[3].float() * 8).round() / 8).clamp(-3, 3).to(dtype)
    if not delta:
        x[4] = x[5] = None
    if mode in (RESIDUAL, MEAN):
        x[3] = None
    return x, [None if t is None else t[:, HEADS] for t in x]


def same_sampled(cache, ref):
    for n in INTS:
        assert getattr(cache, n).cpu().tolist() == getattr(ref, n), n
    for n in FLOATS:
        got, want = getattr(cache, n)[:, HEADS].double().cpu(), getattr(ref, n)
        assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max().clamp_min(1.0)), n


@pytest.mark.parametrize("shape", ["long", "short"])
@pytest.mark.parametrize("d,dtype,delta,mode,topk", [
    (128, torch.bfloat16, True, GRM, 0), (128, torch.float32, False, GRM, 0), (64, torch.bfloat16, False, GRM, 0),
    (128, torch.bfloat16, False, SSC, 4), (128, torch.float32, True, SSC, 30), (64, torch.float32, True, SSC, 4),
    (128, torch.bfloat16, True, MEAN, 0), (32, torch.bfloat16, True, GRM, 0), (16, torch.float32, True, SSC, 3),
    (16, torch.bfloat16, False, RESIDUAL, 0)])
def test_steps(d, dtype, delta, mode, topk, shape):
    segs = SHAPES[shape]
    cache, ref, gen, rng = sampled(d, 6, segs, d + topk, mode == SSC)
    B = len(segs)
    for _ in range(3):
        x, few = inputs(gen, B, 1, d, dtype, delta, mode)
        x, few = ([None if t is None else t[:, :, 0].contiguous() for t in z] for z in (x, few))
        slots = rng.sample(range(B), B)
        slots[rng.randrange(B)] = -1
        q, k, v, u, la, be = (gpu(t) for t in x)
        y = torch.full((B, H, d), 7.0, dtype=dtype, device="cuda")
        mcl.mc_decode_step_paged(cache, q, k, v, u, mode, topk, log_alpha=la, beta=be, slots=i32(slots), y=y)
        want = ref.step(*few, slots, mode, topk)
        for b in range(B):
            if b in want:
                near(y[b, HEADS], want[b], TOL[dtype])
            else:
                assert (y[b] == 7.0).all()
        same_sampled(cache, ref)
    assert ref.status == [0]


@pytest.mark.parametrize("shape", ["long", "short"])
@pytest.mark.parametrize("d,dtype,delta,mode,topk,T,tree,C", [
    (128, torch.bfloat16, False, GRM, 0, 16, "tree", 48), (128, torch.bfloat16, True, GRM, 0, 64, "tree", 48),
    (128, torch.bfloat16, True, GRM, 0, 33, "chain", 5), (64, torch.bfloat16, True, GRM, 0, 64, "tree", 48),
    (64, torch.bfloat16, False, GRM, 0, 16, "chain", 7), (128, torch.bfloat16, True, MEAN, 0, 40, "tree", 48),
    (64, torch.bfloat16, True, RESIDUAL, 0, 9, "star", 48), (128, torch.bfloat16, True, GRM, 0, 1, "chain", 48),
    (128, torch.bfloat16, True, SSC, 4, 16, "tree", 48), (128, torch.float32, True, GRM, 0, 32, "tree", 48),
    (64, torch.float32, False, SSC, 4, 12, "tree", 48), (32, torch.bfloat16, True, GRM, 0, 16, "tree", 48),
    (16, torch.float32, True, GRM, 0, 5, "tree", 48)])
def test_drafts(d, dtype, delta, mode, topk, T, tree, C, shape):
    segs = SHAPES[shape]
    cache, ref, gen, rng = sampled(d, C, segs, d + T, mode == SSC)
    B = len(segs)
    x, few = inputs(gen, B, T, d, dtype, delta, mode)
    parent, slots = draft(rng, B, T, tree), rng.sample(range(B), B)
    slots[rng.randrange(B)] = -1
    count = [T if rng.random() < 0.5 else rng.randint(1, T) for _ in range(B)]
    q, k, v, u, la, be = (gpu(t) for t in x)
    y = torch.full((B, H, T, d), 7.0, dtype=dtype, device="cuda")
    run = lambda y: mcl.mc_decode_tree(cache, q, k, v, u, i32(parent), mode, topk, log_alpha=la, beta=be, count=i32(count),  # noqa: E731
                                       slots=i32(slots), y=y)
    run(y)
    assert torch.equal(run(torch.full_like(y, 7.0)), y)  # bit for bit the same again
    want = ref.tree(*few, parent, count, slots, mode, topk)
    got = y[:, HEADS].float().cpu()
    for b in range(B):
        rows = [j for (bb, j) in want if bb == b]
        assert (y[b][:, [j for j in range(T) if j not in rows]] == 7.0).all()
        if rows:
            near(got[b][:, rows], torch.stack([want[b, j] for j in rows], 1), TOL[dtype])
    same_sampled(cache, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", [GRM, MEAN])
def test_drafts_lose_no_bits_but_the_output_s(d, mode):
    """Memories and queries of one sign, where errors of one sign add up.  An output is fp32's within 1e-5 of its size -- its
    products are within 2^-18 = 4e-6, its weights and sums much closer -- and rounded to bf16 once: off by at most
    2^-8 of itself.  On average the rounding is off by nothing: of n outputs with errors evenly spread up to 2^-8 either
    way the mean is within 2^-8 / sqrt(3 n), and with five times that and 1e-5 the bound is 6e-5 for n = 1e5."""
    cache, ref, gen, rng = sampled(d, 48, LONG, 3 * d, False)
    for n in ("pages", "online", "kbar", "ksum"):
        getattr(cache, n).abs_()
        getattr(ref, n).abs_()
    B, T = len(LONG), 33
    x, few = inputs(gen, B, T, d, torch.bfloat16, False, mode)
    for i in (0, 1, 2):
        x[i].abs_()
        few[i] = x[i][:, HEADS]
    q, k, v, u, la, be = (gpu(t) for t in x)
    parent = draft(rng, B, T, "tree")
    y = mcl.mc_decode_tree(cache, q, k, v, u, i32(parent), mode)
    want = ref.tree(*few, parent, None, None, mode, 0)
    want = torch.stack([torch.stack([want[b, j] for j in range(T)], 1) for b in range(B)])
    got = y[:, HEADS].double().cpu()
    assert (want > 0).all()
    off = (got - want) / want
    assert float(off.abs().max()) <= 2 ** -8 + 1e-5
    assert off.numel() > 1e5 / 2 and abs(float(off.mean())) <= 5 * 2 ** -8 / (3 * off.numel()) ** 0.5 + 1e-5


@pytest.mark.parametrize("d", [64, 128])
def test_drafts_of_what_is_not_finite(d):
    """An infinity, a NaN (one that differs from an infinity in its last bit) and numbers at the type's ends in cached memories:
    outputs are what the products and sums in 64 bits are, where those fit; the other sequences' are untouched."""
    cache, ref, gen, rng = sampled(d, 48, [6, 5, 7, 4], d, False)
    B, T = 4, 20
    cache.pages.mul_(0.125)
    ref.pages.mul_(0.125)
    x, few = inputs(gen, B, T, d, torch.bfloat16, False, MEAN)
    for i in (0,):
        x[i].abs_().clamp_min_(2.0 ** -8)
        few[i] = x[i][:, HEADS]
    last_nan = torch.tensor([0x7f800001], dtype=torch.int32).view(torch.float32)
    odd = [(0, float("inf")), (1, float("nan")), (2, last_nan.item())]
    for b, value in odd:
        p = ref.table[ref.row[b]][2]
        if b == 2:
            cache.pages.view(torch.int32)[p, :, 3, 5] = 0x7f800001
        else:
            cache.pages[p, :, 3, 5] = value
        ref.pages[p, :, 3, 5] = float("nan") if b else value
    p = ref.table[ref.row[3]][1]
    cache.pages[p, :, 7, 4], ref.pages[p, :, 7, 4] = 3.4e38, float(torch.tensor(3.4e38))
    q, k, v, u, la, be = (gpu(t) for t in x)
    parent = draft(rng, B, T, "star")
    y = mcl.mc_decode_tree(cache, q, k, v, None, i32(parent), MEAN)
    want = ref.tree(*few, parent, None, None, MEAN, 0)
    got = y[:, HEADS].double().cpu()
    for (b, j), w in want.items():
        rest = torch.ones(d, dtype=torch.bool)
        rest[7 if b == 3 else 3] = False
        near(got[b, :, j][:, rest], w[:, rest], 1e-2)
        if b == 0:
            assert (got[b, :, j, 3] == float("inf")).all()
        elif b < 3:
            assert torch.isnan(got[b, :, j, 3]).all()
        else:
            assert float((got[b, :, j, 7] / w[:, 7] - 1).abs().max()) <= 2 ** -8 + 1e-4


@pytest.mark.parametrize("d,T,dtype", [(128, 9, torch.bfloat16), (64, 9, torch.bfloat16), (128, 2, torch.bfloat16), (128, 3, torch.float32)])
def test_a_full_batch_of_drafts(d, T, dtype):
    """1024 sequences: the most rows that a call takes, all of whose places a CTA holds in shared memory."""
    S, C = 1024, 4
    gen, rng = seeded(d + T)
    segs = [rng.randrange(3) for _ in range(S)]
    n_max = 700 if T < 9 else 4  # (room for so much that a few nodes take every kernel)
    ref = Ref(S, 1, d, C, n_max, sum(segs) + 8).fill(segs, [rng.randrange(C) for _ in range(S)], gen, rng)
    cache = ref.to(mcl.PagedCache(S, 1, d, C, n_max, ref.P))
    x = tokens(gen, S, 1, T, d, dtype)
    parent = draft(rng, S, T, "tree")
    y = torch.full((S, 1, T, d), 7.0, dtype=dtype, device="cuda")
    q, k, v, u, la, be = (gpu(t) for t in x)
    mcl.mc_decode_tree(cache, q, k, v, u, i32(parent), GRM, log_alpha=la, beta=be, y=y)
    want = ref.tree(*x, parent, None, None, GRM, 0)
    near(y, torch.stack([torch.stack([want[b, j] for j in range(T)], 1) for b in range(S)]), TOL[dtype])
    assert cache.status.item() == 0
