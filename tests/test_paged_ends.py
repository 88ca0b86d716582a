"""Where a sequence's table ends, in the 64-bit form: a draft reads the segments that its path completes whether or not they find a
page; steps lose those past the table's end."""
import pytest
import torch

from paged_ref import GRM, MEAN, SSC, TABLE_FULL, Ref, draft, seeded, tokens


@pytest.mark.parametrize("mode,topk", [(GRM, 0), (SSC, 2), (MEAN, 0)])
@pytest.mark.parametrize("n_max,P", [(3, 30), (12, 3)])
def test_a_draft_reads_what_steps_with_room_would(n_max, P, mode, topk):
    T, H, d, C = 9, 1, 16, 2
    def made(n_max, P):
        gen, rng = seeded(6)
        ref = Ref(1, H, d, C, n_max, 30).fill([3], [1], gen, rng)  # three segments: the table of three is full
        if P < 30:
            ref.refs = [max(r, int(p not in ref.table[0])) for p, r in enumerate(ref.refs)]  # no page is free
        return ref, gen, rng
    ref, gen, rng = made(n_max, P)
    x = tokens(gen, 1, H, T, d, torch.float64)
    parent = draft(rng, 1, T, "chain")
    got = ref.tree(*x, parent, None, None, mode, topk)
    roomy, _, _ = made(12, 30)
    same = short = 0
    for j in range(T):
        tok = [t[:, :, j] for t in x]
        y, lost = roomy.step(*tok, None, mode, topk)[0], ref.step(*tok, None, mode, topk)[0]
        assert (y - got[0, j]).abs().max() < 1e-12
        same += bool((lost - y).abs().max() < 1e-12)
        short += bool((lost - y).abs().max() > 1e-6)
    assert roomy.status == [0] and ref.status != [0] and same >= 1 and short >= 1
