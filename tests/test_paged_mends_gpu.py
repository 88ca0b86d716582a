"""Calls of the paged cache that the other tests' sizes do not reach.  Tolerances as in test_paged_gpu.py: of an output's largest
value 1e-4 with fp32 inputs, 1e-2 with bf16 ones; what is copied or counted is equal."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from paged_ref import GRM, Ref, draft, seeded, tokens
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
