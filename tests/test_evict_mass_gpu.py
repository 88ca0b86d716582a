"""The gate weights of an evicting cache over long streams, against their sums in 64 bits."""
import math

import pytest
import torch

import memory_caching_linear_gb300 as mcl
from delta_ref import GRM

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from memory_caching_linear_gb300 import build
    build.build()
    mcl.load_library()


def stream(start, gates, steps):
    """A cache whose slots hold the masses `start` and gather the same `gates` at each of `steps` tokens, the last of
    which completes a segment."""
    n, d = len(start), 16
    cache = mcl.EvictingCache(1, 1, d, steps, n, protect=0)
    cache.slot_seg.copy_(torch.arange(n).view(1, 1, n))
    cache.mass.copy_(torch.tensor(start).view(1, 1, n))
    cache.kbar[0, 0, :, 0] = torch.tensor([math.log(g / (1 - sum(gates))) for g in gates])  # online score 0
    cache.t = n * steps
    zero, u = torch.zeros(1, 1, d, device="cuda"), torch.zeros(1, 1, d, device="cuda")
    u[..., 0] = 1.0
    for _ in range(steps - 1):
        mcl.mc_decode_step_evict(cache, zero, zero, zero, u, GRM)
    mass = cache.mass[0, 0].double().cpu()
    mcl.mc_decode_step_evict(cache, zero, zero, zero, u, GRM)
    return mass, cache.slot_seg[0, 0].tolist()


def last_place(x):
    return 2.0 ** (math.floor(math.log2(x)) - 23)


@pytest.mark.parametrize("start", [0.0, 40.0, 2.0 ** 16, 1e6, 2.0 ** 20, 2.0 ** 24])
def test_small_gates_count_in_large_masses(start):
    """The multiples of the golden ratio leave the share of 2000 of them below any bound at most 6 off what it ought to be
    (their discrepancy is below 0.67 log2(n) / n), so a mass is within 8 last places; the gates themselves are fp32,
    2000 of them off by 2^-21 each at most."""
    steps, gates = 2001, [0.2, 0.03, 0.004, 0.0005]
    mass, _ = stream([start] * 4, gates, steps)
    for m, g in zip(mass.tolist(), gates):
        want = start + (steps - 1) * g
        assert abs(m - want) <= 8 * last_place(want) + (steps - 1) * 2.0 ** -21 * g, (m, want)


def test_the_segment_with_the_least_mass_goes():
    """Just below 2^20 a gate of 0.04 would always be rounded up to 0.0625, and above it one of 0.05 down to nothing."""
    steps = 400
    start, gates = [1048576.0, 1048574.0], [0.05, 0.04]
    final = [s + steps * g for s, g in zip(start, gates)]  # 1048596 and 1048590
    assert final[0] > final[1] + 5
    _, slots = stream(start, gates, steps)
    assert slots == [0, 2]


def test_equal_masses_with_equal_gates_stay_equal():
    mass, slots = stream([1e6] * 3, [0.01] * 3, 300)
    assert len(set(mass.tolist())) == 1 and slots == [3, 1, 2]  # and then the oldest goes
