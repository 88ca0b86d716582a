"""Decoding with eviction by accumulated gate weight, and the compaction of a prefill, against their 64-bit forms.

Tolerances as the forward's: y 1e-4 (fp32) and 1e-2 (bf16) of the largest value; states, key means and masses 1e-4
(fp32 sums of exact inputs).  Which segment leaves is compared exactly: the inputs keep the masses apart."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, MEAN, RESIDUAL, SOUP, SSC, Slots, compact, forward, make_delta_inputs

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-4, "bf16": 1e-2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from memory_caching_linear_gb300 import build
    build.build()
    mcl.load_library()


def rel(got, ref):
    ref = ref.double()
    scale = float(ref.abs().max())
    return float((got.double().cpu() - ref).abs().max()) / (scale if scale > 0 else 1.0)


def same_cache(cache, ref):
    assert torch.equal(cache.slot_seg.cpu().long(), ref.slot_seg)
    for name in ("states", "kbar", "mass", "online", "ksum"):
        assert rel(getattr(cache, name), getattr(ref, name)) <= 1e-4, name


def run(x, C, mode, topk, n_max, protect, delta, cache=None, ref=None, first=0):
    xd = [t.cuda() for t in x]
    B, H, L, d = x[0].shape
    cache = cache or mcl.EvictingCache(B, H, d, C, n_max, protect=protect)
    ref = ref or Slots(B, H, d, C, n_max, protect)
    got, want = [], []
    for j in range(first, L):
        tok = [t[:, :, j].contiguous() for t in xd]
        kw = dict(log_alpha=tok[4], beta=tok[5]) if delta else {}
        got.append(mcl.mc_decode_step_evict(cache, *tok[:4], mode, topk, **kw))
        want.append(ref.step(*(t[:, :, j] for t in x[:4]), mode, topk, *((t[:, :, j] for t in x[4:]) if delta else ())))
    return torch.stack(got, 2), torch.stack(want, 2), cache, ref


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SOUP, 0), (SSC, 2), (SSC, 0)])
@pytest.mark.parametrize("d,C,L,n_max,protect,dtype", [
    (16, 4, 60, 4, 1, "f32"), (32, 5, 64, 3, 0, "bf16"), (64, 3, 50, 5, 2, "bf16"), (128, 4, 44, 1, 0, "f32"),
    (128, 1, 90, 64, 3, "bf16"), (64, 2, 100, 33, 32, "f32")])
def test_decode_with_eviction(d, C, L, n_max, protect, dtype, mode, topk, delta):
    x = make_delta_inputs(1, 3, L, d, C, d + L + n_max, dtype)
    got, want, cache, ref = run(x, C, mode, topk, n_max, protect, delta)
    assert rel(got, want) <= TOL[dtype]
    same_cache(cache, ref)


def test_equal_masses_drive_out_the_oldest():
    """Key means of zero give every cached segment the same gate: newer ones have gathered less, until all are equal."""
    B, H, d, C, n = 1, 1, 16, 1, 4
    cache = mcl.EvictingCache(B, H, d, C, n, protect=0)
    cache.slot_seg.copy_(torch.tensor([[[6, 3, 5, 4]]]))
    cache.t = 7
    z = torch.zeros(B, H, d, device="cuda")
    mcl.mc_decode_step_evict(cache, z, z, z, z, GRM)
    assert cache.slot_seg.cpu().tolist() == [[[6, 7, 5, 4]]] and cache.mass[0, 0, 1] == 0
    assert torch.allclose(cache.mass[0, 0, [0, 2, 3]], torch.full((3,), 0.2, device="cuda"))
    cache.mass.zero_()
    cache.protect = 3  # the newest three of 6, 7, 5, 4 stay
    mcl.mc_decode_step_evict(cache, z, z, z, z, GRM)
    assert cache.slot_seg.cpu().tolist() == [[[6, 7, 5, 8]]]


def test_empty_slots_are_filled_first_and_never_read():
    B, H, d, C = 1, 2, 32, 2
    x = make_delta_inputs(B, H, 6, d, C, 5, "f32")
    cache = mcl.EvictingCache(B, H, d, C, 5, protect=1)
    cache.states.fill_(float("nan"))
    cache.kbar.fill_(float("nan"))
    cache.online.fill_(float("nan"))
    cache.ksum.fill_(float("nan"))
    got, want, cache, ref = run(x, C, GRM, 0, 5, 1, False, cache=cache)
    assert rel(got, want) <= TOL["f32"]
    assert cache.slot_seg.cpu().tolist() == [[[0, 1, 2, -1, -1]] * H]
    assert torch.isnan(cache.states[:, :, 3:]).all()


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SOUP, 0), (SSC, 1), (SSC, 3)])
@pytest.mark.parametrize("d,C,L,n_max,protect,dtype", [
    (16, 8, 100, 4, 1, "f32"), (32, 13, 200, 6, 0, "bf16"), (64, 16, 128, 3, 3, "bf16"), (128, 9, 333, 20, 2, "f32"),
    (64, 3, 250, 64, 1, "bf16"), (128, 32, 320, 5, 1, "bf16"), (64, 50, 30, 3, 1, "f32"), (64, 64, 128, 8, 1, "bf16"),
    (128, 2, 300, 33, 1, "bf16")])
def test_compact(d, C, L, n_max, protect, dtype, mode, topk):
    x = make_delta_inputs(2, 2, L, d, C, d + L, dtype)
    gen = torch.Generator().manual_seed(1)
    st = torch.randn(2, 2, -(-L // C), d, d, generator=gen)
    ref, mass = compact(x[1], x[3], st, C, mode, topk, n_max, protect)
    cache = mcl.EvictingCache(2, 2, d, C, n_max, protect=protect)
    for t in (cache.states, cache.kbar, cache.mass, cache.online, cache.ksum):
        t.fill_(float("nan"))
    got = mcl.mc_cache_compact(cache, x[1].cuda(), x[3].cuda(), st.cuda(), mode, topk)
    assert mcl.mc_check_device() == mcl.MC_OK
    assert cache.t == L and rel(got, mass) <= 1e-4
    same_cache(cache, ref)
    twice = mcl.EvictingCache(2, 2, d, C, n_max, protect=protect)
    again = mcl.mc_cache_compact(twice, x[1].cuda(), x[3].cuda(), st.cuda(), mode, topk)
    assert torch.equal(again, got) and torch.equal(twice.slot_seg, cache.slot_seg)


def test_more_segments_than_a_block_of_scores():
    x = make_delta_inputs(1, 1, 700, 64, 4, 77, "bf16")
    st = torch.randn(1, 1, 175, 64, 64, generator=torch.Generator().manual_seed(2))
    for mode, topk in ((GRM, 0), (SSC, 8)):
        ref, mass = compact(x[1], x[3], st, 4, mode, topk, 40, 2)
        cache = mcl.EvictingCache(1, 1, 64, 4, 40, protect=2)
        assert rel(mcl.mc_cache_compact(cache, x[1].cuda(), x[3].cuda(), st.cuda(), mode, topk), mass) <= 1e-4
        same_cache(cache, ref)


@pytest.mark.parametrize("delta", [False, True])
def test_prefill_compact_decode(delta):
    """The three together: a prefill of more segments than slots, its compaction, and decoding over segment ends."""
    B, H, L, P, d, C, n_max = 1, 2, 220, 170, 64, 16, 6
    x = make_delta_inputs(B, H, L, d, C, 13, "bf16")
    head = [t[:, :, :P].contiguous() for t in x]
    if delta:
        _, st64 = forward(*head, C, GRM)
        _, st = mcl.mc_forward_delta(*(t.cuda() for t in head), C, GRM)
    else:
        q, k, v = (t.double() for t in head[:3])
        st64 = torch.stack([v[:, :, n * C:(n + 1) * C].transpose(2, 3) @ k[:, :, n * C:(n + 1) * C] for n in range(-(-P // C))], 2)
        _, st = mcl.mc_forward(*(t.cuda() for t in head[:4]), C, GRM)
    ref, _ = compact(head[1], head[3], st64, C, GRM, 0, n_max, 1)
    prompt = mcl.EvictingCache(B, H, d, C, n_max)
    mcl.mc_cache_compact(prompt, head[1].cuda(), head[3].cuda(), st, GRM)
    same_cache(prompt, ref)
    cache = mcl.EvictingCache(B, H, d, C, n_max).copy_(prompt)
    got, want, cache, ref = run(x, C, GRM, 0, n_max, 1, delta, cache=cache, ref=ref, first=P)
    assert rel(got, want) <= TOL["bf16"]
    same_cache(cache, ref)
    assert prompt.t == P  # the prompt's cache is untouched: a second continuation is the same
    again, _, _, _ = run(x, C, GRM, 0, n_max, 1, delta, cache=cache.copy_(prompt), ref=Slots(B, H, d, C, n_max, 1), first=P)
    assert torch.equal(again, got)


def test_step_in_a_graph_and_on_a_side_stream():
    B, H, d, C, n = 1, 2, 64, 50, 4
    x = [t[:, :, 0].contiguous().cuda() for t in make_delta_inputs(B, H, 4, d, C, 3, "bf16")]
    def fresh():
        c = mcl.EvictingCache(B, H, d, C, n)
        g = torch.Generator("cuda").manual_seed(4)
        for t in (c.states, c.kbar, c.online, c.ksum):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        c.slot_seg.copy_(torch.tensor([3, 0, 2, 1]))
        c.t = 4 * C + 7
        return c
    a, b = fresh(), fresh()
    want = mcl.mc_decode_step_evict(a, *x[:4], GRM, log_alpha=x[4], beta=x[5])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = mcl.mc_decode_step_evict(b, *x[:4], GRM, log_alpha=x[4], beta=x[5])
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(a.mass, b.mass) and torch.equal(a.online, b.online)
    c = fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mcl.mc_decode_step_evict(c, *x[:4], GRM, log_alpha=x[4], beta=x[5])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(a.mass, c.mass)


@pytest.mark.parametrize("mode", [RESIDUAL, MEAN])
def test_constant_gates_are_refused(mode):
    z = torch.zeros(1, 1, 16, device="cuda")
    cache = mcl.EvictingCache(1, 1, 16, 4, 2)
    with pytest.raises(mcl.MCError) as e:
        mcl.mc_decode_step_evict(cache, z, z, z, z, mode)
    assert e.value.status == mcl.MC_ERR_MODE and cache.t == 0


def test_offsets_past_32_bits():
    """More than 2^31 numbers in the cache and in the prefill's states: copies of one head, the last as the first."""
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    BH, d, C, n_max = 8400, 64, 4, 63
    L = 66 * C + 2
    assert BH * n_max * d * d > 2**31
    one = make_delta_inputs(1, 1, L + 4, d, C, 91, "bf16")
    st1 = torch.randn(1, 1, 67, d, d, generator=torch.Generator().manual_seed(3))
    head = [t[:, :, :L].contiguous() for t in one]
    ref, mass = compact(head[1], head[3], st1, C, GRM, 0, n_max, 2)
    cache = mcl.EvictingCache(1, BH, d, C, n_max, protect=2)
    wide = lambda t: t.cuda().expand(1, BH, *t.shape[2:]).contiguous()
    got = mcl.mc_cache_compact(cache, wide(head[1]), wide(head[3]), wide(st1), GRM)
    assert torch.equal(got[:, 0], got[:, -1]) and rel(got[:, :1], mass) <= 1e-4
    for j in range(L, L + 4):  # over a segment's end
        tok = [t[:, :, j].contiguous() for t in one]
        w = [t.cuda().expand(1, BH, *t.shape[2:]).contiguous() for t in tok]
        y = mcl.mc_decode_step_evict(cache, *w[:4], GRM, log_alpha=w[4], beta=w[5])
        want = ref.step(*tok[:4], GRM, 0, *tok[4:])
        assert torch.equal(y[:, 0], y[:, -1]) and rel(y[:, :1], want) <= TOL["bf16"]
    assert torch.equal(cache.slot_seg[:, 0], cache.slot_seg[:, -1]) and torch.equal(cache.states[:, 0], cache.states[:, -1])
    assert torch.equal(cache.slot_seg[:, :1].cpu().long(), ref.slot_seg) and rel(cache.states[:, :1], ref.states) <= 1e-4


def test_caches_of_different_shapes_are_not_copied():
    a = mcl.EvictingCache(1, 2, 32, 4, 3)
    for b in (mcl.EvictingCache(1, 1, 32, 4, 3), mcl.EvictingCache(1, 2, 32, 4, 2), mcl.EvictingCache(1, 2, 32, 5, 3)):
        with pytest.raises(ValueError):
            a.copy_(b)
