"""Calls of the paged cache's operators that are refused before they touch a device."""
import ctypes

import pytest
import torch

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild

FAKE = 1 << 20  # an aligned address that is never read
PTRS = ("pages", "kbar", "refs", "online", "ksum", "table", "pos", "row", "status", "work")


@pytest.fixture(scope="module")
def lib():
    mcbuild.build()
    return mcl.load_library()


def cache(**kw):
    a = {n: FAKE for n in PTRS} | dict(n_pages=8, n_seqs=4, H=2, d=16, seg_len=4, n_max=4) | kw
    return ctypes.byref(mcl._CPagedCache(*a.values()))


def step(lib, c=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, u=FAKE, la=FAKE, be=FAKE, slots=FAKE, B=2, mode=1, topk=0, y=FAKE) | kw
    return lib.mc_decode_step_paged(c or cache(), *a.values(), 1, None)


def tree(lib, c=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, u=FAKE, la=FAKE, be=FAKE, parent=FAKE, count=FAKE, slots=FAKE, B=2, T=3, mode=1, topk=0, y=FAKE) | kw
    return lib.mc_decode_tree(c or cache(), *a.values(), 1, None)


def accept(lib, c=None, **kw):
    a = dict(k=FAKE, v=FAKE, la=FAKE, be=FAKE, parent=FAKE, last=FAKE, slots=FAKE, B=2, T=3) | kw
    return lib.mc_tree_accept(c or cache(), *a.values(), 1, None)


def fork(lib, c=None, src=FAKE):
    return lib.mc_pages_fork(c or cache(), src, None)


def compact(lib, c=None, other=None):
    return lib.mc_pages_compact(other or cache(**{n: 2 * FAKE for n in PTRS}), c or cache(), None)


def load(lib, c=None, **kw):
    a = dict(slot=0, k=FAKE, states=FAKE, L=10) | kw
    return lib.mc_pages_load(c or cache(), *a.values(), 1, None)


@pytest.mark.parametrize("call", [step, tree, accept, fork, compact, load])
def test_caches(lib, call):
    for bad in (dict(d=24), dict(d=256), dict(H=0), dict(seg_len=0), dict(n_seqs=0), dict(n_seqs=1025), dict(n_max=0),
                dict(n_max=1025), dict(n_pages=0), dict(n_pages=(1 << 20) + 1), dict(H=1 << 21)):
        assert call(lib, cache(**bad)) == mcl.MC_ERR_SHAPE, bad
    for n in PTRS:
        assert call(lib, cache(**{n: None})) == mcl.MC_ERR_NULL, n
        off = 8 if n in ("pages", "kbar", "online", "ksum", "work") else 2
        assert call(lib, cache(**{n: FAKE + off})) == mcl.MC_ERR_ALIGN, n


def test_no_cache(lib):
    assert lib.mc_pages_fork(None, FAKE, None) == mcl.MC_ERR_NULL
    assert lib.mc_pages_compact(None, cache(), None) == mcl.MC_ERR_NULL
    assert lib.mc_pages_compact(cache(), None, None) == mcl.MC_ERR_NULL


@pytest.mark.parametrize("call", [step, tree])
def test_reading_calls(lib, call):
    for n in ("q", "k", "v", "u", "y"):
        assert call(lib, **{n: None}) == mcl.MC_ERR_NULL, n
        assert call(lib, **{n: FAKE + 8}) == mcl.MC_ERR_ALIGN, n
    assert call(lib, slots=FAKE + 2) == mcl.MC_ERR_ALIGN and call(lib, la=FAKE + 1) == mcl.MC_ERR_ALIGN
    assert call(lib, la=None) == mcl.MC_ERR_NULL and call(lib, be=None) == mcl.MC_ERR_NULL  # one without the other
    assert call(lib, B=0) == mcl.MC_ERR_SHAPE and call(lib, B=5) == mcl.MC_ERR_SHAPE
    assert call(lib, mode=5) == mcl.MC_ERR_MODE and call(lib, mode=-1) == mcl.MC_ERR_MODE
    assert call(lib, mode=mcl.MC_SSC, topk=-1) == mcl.MC_ERR_TOPK
    for mode in (mcl.MC_RESIDUAL, mcl.MC_MEAN):  # no router: u may be absent (the misaligned y stops the call)
        assert call(lib, mode=mode, u=None, y=FAKE + 4) == mcl.MC_ERR_ALIGN
    assert call(lib, la=FAKE + 2, be=FAKE + 2, slots=None, y=FAKE + 4) == mcl.MC_ERR_ALIGN  # the gates begin at any element


def test_drafts(lib):
    for call in (tree, accept):
        assert call(lib, T=0) == mcl.MC_ERR_SHAPE and call(lib, T=65) == mcl.MC_ERR_SHAPE and call(lib, B=5) == mcl.MC_ERR_SHAPE
        assert call(lib, parent=None) == mcl.MC_ERR_NULL and call(lib, parent=FAKE + 1) == mcl.MC_ERR_ALIGN
    assert tree(lib, T=1, parent=None, y=FAKE + 4) == mcl.MC_ERR_ALIGN
    assert tree(lib, count=FAKE + 2) == mcl.MC_ERR_ALIGN
    assert accept(lib, last=None) == mcl.MC_ERR_NULL and accept(lib, last=FAKE + 2) == mcl.MC_ERR_ALIGN
    assert accept(lib, k=None) == mcl.MC_ERR_NULL and accept(lib, v=FAKE + 8) == mcl.MC_ERR_ALIGN
    assert accept(lib, la=None) == mcl.MC_ERR_NULL


def test_pools(lib):
    assert fork(lib, src=None) == mcl.MC_ERR_NULL and fork(lib, src=FAKE + 2) == mcl.MC_ERR_ALIGN
    far = {n: 2 * FAKE for n in PTRS}
    for other in (dict(H=3), dict(d=32), dict(seg_len=5), dict(n_seqs=3), dict(n_max=3)):
        assert compact(lib, other=cache(**far | other)) == mcl.MC_ERR_SHAPE, other
    assert compact(lib, other=cache()) == mcl.MC_ERR_SHAPE  # a cache into itself
    for bad in (dict(slot=-1), dict(slot=4), dict(L=0), dict(L=(1 << 30) + 1), dict(L=20)):  # 20 tokens: five segments of four
        assert load(lib, **bad) == mcl.MC_ERR_SHAPE, bad
    assert load(lib, L=19, k=FAKE + 8) == mcl.MC_ERR_ALIGN
    assert load(lib, k=None) == mcl.MC_ERR_NULL and load(lib, states=FAKE + 4) == mcl.MC_ERR_ALIGN


def test_work_bytes(lib):
    """Tickets of every head and one more, then 152 ranges' and every head's partial reads, then the online memories'."""
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    for S, H, d in ((1, 1, 16), (24, 16, 128), (1024, 7, 64)):
        assert lib.mc_paged_work_bytes(S, H, d) == up(4 * (S * H + 1)) + up(4 * (152 + S * H) * (d + 2)) + up(4 * S * H * (d + 1))
    assert lib.mc_paged_work_bytes(0, 1, 16) == 0 and lib.mc_paged_work_bytes(1025, 1, 16) == 0 and lib.mc_paged_work_bytes(1, 0, 16) == 0


def test_the_binding(lib):
    c = mcl.PagedCache(3, 2, 16, 4, 5, 7, device="cpu")
    assert c.table.tolist() == [[-1] * 5] * 3 and c.row.tolist() == [0, 1, 2] and c.refs.tolist() == [0] * 7
    with pytest.raises(AttributeError):
        c.pages = torch.zeros(1)
    with pytest.raises(ValueError):
        mcl.PagedCache(3, 2, 16, 0, 5, 7, device="cpu")
    z = torch.zeros(2, 2, 16)
    with pytest.raises(ValueError):  # not on the GPU
        mcl.mc_decode_step_paged(c, z, z, z, z, mcl.MC_GRM)
    with pytest.raises(ValueError):
        mcl.mc_decode_tree(c, z, z, z, z, torch.zeros(2, 1), mcl.MC_GRM)
    with pytest.raises(ValueError):
        mcl.mc_pages_fork(c, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        mcl.mc_pages_fork(mcl.DecodeCache(1, 1, 16, 4, 2, device="cpu"), torch.zeros(3, dtype=torch.int32))
    c.check()
    c.status.fill_(mcl.MC_PAGES_NONE_FREE)
    with pytest.raises(RuntimeError, match="no free page"):
        c.check()
    c.check()
