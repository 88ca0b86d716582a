"""Copies of a paged cache, as the other caches can be copied."""
import copy
import ctypes
import pickle

import pytest
import torch

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild

NAMES = ("pages", "kbar", "refs", "online", "ksum", "table", "pos", "row", "status")


@pytest.fixture(scope="module", autouse=True)
def lib():
    mcbuild.build()


@pytest.mark.parametrize("how", [copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_a_copy_has_tensors_of_its_own(how):
    c = mcl.PagedCache(3, 2, 16, 4, 5, 7, device="cpu")
    c.pages.normal_()
    c.table[1, 2], c.pos[1], c.refs[4] = 4, 13, 1
    d = how(c)
    for n in NAMES:
        assert torch.equal(getattr(c, n), getattr(d, n)) and getattr(c, n).data_ptr() != getattr(d, n).data_ptr(), n
        assert getattr(d._c, n) == getattr(d, n).data_ptr(), n  # what the library is given
    assert d._c.work == d._t["work"].data_ptr() != c._c.work and d._ref == ctypes.addressof(d._c) != c._ref
    for n in ("n_pages", "n_seqs", "H", "d", "seg_len", "n_max"):
        assert getattr(d._c, n) == getattr(c._c, n) == getattr(d, n)
    assert d.device == c.device
    d.pos.fill_(7)
    assert c.pos.tolist() == [0, 13, 0]
    with pytest.raises(AttributeError):
        d.pages = torch.zeros(1)


def test_a_shallow_copy_shares_them():
    c = mcl.PagedCache(2, 1, 16, 4, 3, 2, device="cpu")
    d = copy.copy(c)
    assert d.pages.data_ptr() == c.pages.data_ptr() == d._c.pages
