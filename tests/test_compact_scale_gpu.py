"""Compaction of prefills of thousands of segments: the masses against the definition in 64 bits, the choice against the
masses, and scratch that grows with the prefill.  Tolerance of the masses as in test_evict_gpu.py, 1e-4 of the largest."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM, SSC

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from memory_caching_linear_gb300 import build
    build.build()
    mcl.load_library()


def prefill(H, L, d, C, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    N = -(-L // C)
    topics = torch.randn(1, H, N, d, device="cuda", generator=g)
    topics /= topics.norm(dim=-1, keepdim=True)
    seg = torch.arange(L, device="cuda") // C
    k = 0.7 * topics[:, :, seg] + torch.randn(1, H, L, d, device="cuda", generator=g) / d ** 0.5
    liked = torch.randint(0, N, (1, H, L, 1), device="cuda", generator=g)
    u = 6 * torch.gather(topics, 2, liked.expand(1, H, L, d)) + torch.randn(1, H, L, d, device="cuda", generator=g) / d ** 0.5
    st = torch.randn(1, H, N, d, d, device="cuda", generator=g)
    return k.to(dtype), u.to(dtype), st


def masses(k, u, C, mode, topk):
    """sum_t g_{t,i} in 64 bits, 512 tokens at a time."""
    _, H, L, d = k.shape
    N = -(-L // C)
    out = torch.zeros(1, H, N, dtype=torch.float64, device="cuda")
    for h in range(H):
        kd, ud = k[0, h].double(), u[0, h].double()
        run = torch.cat([torch.zeros(1, d, dtype=torch.float64, device="cuda"), kd.cumsum(0)])
        begin = torch.arange(N, device="cuda") * C
        end = torch.clamp(begin + C, max=L)
        kbar = (run[end] - run[begin]) / (end - begin)[:, None]
        for a in range(0, L, 512):
            t = torch.arange(a, min(L, a + 512), device="cuda")
            s = t // C
            r = ud[t] @ kbar.T
            r = r.masked_fill(torch.arange(N, device="cuda")[None] >= s[:, None], float("-inf"))
            if mode == SSC:
                best = torch.topk(r, topk, -1).indices
                r = torch.full_like(r, float("-inf")).scatter(-1, best, torch.gather(r, -1, best))
            on = (ud[t] * (run[t + 1] - run[s * C]) / (t + 1 - s * C)[:, None]).sum(-1, keepdim=True)
            out[0, h] += torch.softmax(torch.cat([r, on], -1), -1)[:, :N].sum(0)
    return out


@pytest.mark.parametrize("H,L,d,C,dtype,mode,topk", [
    (2, 40001, 16, 5, torch.bfloat16, GRM, 0), (1, 70001, 64, 37, torch.bfloat16, GRM, 0), (1, 66000, 128, 600, torch.bfloat16, GRM, 0),
    (1, 33000, 32, 3, torch.bfloat16, SSC, 4), (1, 33001, 128, 100, torch.float32, GRM, 0), (1, 17000, 16, 2, torch.float32, SSC, 2)])
def test_masses_of_long_prefills(H, L, d, C, dtype, mode, topk):
    """More tiles of tokens than a head has partial sums (512, or 256 for d = 16)."""
    k, u, st = prefill(H, L, d, C, dtype, L)
    n_max, protect = 24, 2
    cache = mcl.EvictingCache(1, H, d, C, n_max, protect=protect)
    got = mcl.mc_cache_compact(cache, k, u, st, mode, topk)
    want = masses(k, u, C, mode, topk)
    assert float((got.double() - want).abs().max()) <= 1e-4 * float(want.max())
    again = mcl.mc_cache_compact(cache, k, u, st, mode, topk)
    assert torch.equal(again, got)
    done = L // C
    for h in range(H):
        rank = sorted(range(done - protect), key=lambda i, m=got[0, h].tolist(): (m[i], i))
        kept = sorted(rank[len(rank) - (n_max - protect):] + list(range(done - protect, done)))
        assert cache.slot_seg[0, h].tolist() == kept
        assert torch.equal(cache.mass[0, h], got[0, h, kept]) and torch.equal(cache.states[0, h], st[0, h, kept])


@pytest.mark.parametrize("dtype,mode,topk", [(torch.bfloat16, GRM, 0), (torch.bfloat16, SSC, 2), (torch.float32, GRM, 0)])
def test_scratch_of_many_segments(dtype, mode, topk):
    """A tile of tokens has no row of sums of its own: with 16384 segments these rows would be several times the prefill."""
    H, L, d, C = 4, 1 << 17, 16, 8
    k, u, st = prefill(H, L, d, C, dtype, 1)
    cache, mass = mcl.EvictingCache(1, H, d, C, 8), torch.empty(1, H, L // C, device="cuda")
    torch.cuda.synchronize()
    assert mcl.mc_trim_scratch() == mcl.MC_OK
    free = torch.cuda.mem_get_info()[0]
    mcl.mc_cache_compact(cache, k, u, st, mode, topk, mass=mass)
    torch.cuda.synchronize()
    used = free - torch.cuda.mem_get_info()[0]
    mcl.mc_trim_scratch()
    # the sums as much as the states, the key means' images 3/4 of that, the key sums, means and scores under 1/4; the
    # pool grows by 32 MiB at a time
    assert used <= 2 * st.numel() * 4 + (32 << 20)
