"""The gated delta memory's and the evicting cache's entry points refuse bad arguments before they touch a device."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild

FAKE = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    mcbuild.build()
    return mcl.load_library()


SHAPE = dict(B=1, H=1, L=64, d=16, seg=16, mode=mcl.MC_GRM, topk=0)
FORWARD = (["q", "k", "v", "u", "la", "be"], ["y", "states"])
BACKWARD = (["q", "k", "v", "u", "la", "be", "dy"], ["dq", "dk", "dv", "du", "dla", "dbe"])


def call(lib, kind, **kw):
    a = dict(SHAPE)
    ins, outs = FORWARD if kind == "forward" else BACKWARD
    a.update({n: FAKE for n in ins + outs})
    a.update(kw)
    fn = lib.mc_forward_delta if kind == "forward" else lib.mc_backward_delta
    return fn(*(a[n] for n in ins), *(a[n] for n in SHAPE), *(a[n] for n in outs), 1, None)


@pytest.mark.parametrize("kind", ["forward", "backward"])
def test_sequence_arguments(lib, kind):
    ins, outs = FORWARD if kind == "forward" else BACKWARD
    for n in ins + outs:
        if n != "states":
            assert call(lib, kind, **{n: None}) == mcl.MC_ERR_NULL, n
        assert call(lib, kind, **{n: FAKE + 8}) == mcl.MC_ERR_ALIGN, n
    for mode in (mcl.MC_RESIDUAL, mcl.MC_MEAN):  # no router: u and du may be absent
        assert call(lib, kind, mode=mode, u=None, q=FAKE + 4, **({"du": None} if kind == "backward" else {})) == mcl.MC_ERR_ALIGN
    for bad in (dict(d=17), dict(d=256), dict(L=0), dict(B=0), dict(H=-1), dict(seg=0), dict(B=1 << 20, H=1 << 10)):
        assert call(lib, kind, **bad) == mcl.MC_ERR_SHAPE, bad
    assert call(lib, kind, mode=7) == mcl.MC_ERR_MODE and call(lib, kind, mode=-1) == mcl.MC_ERR_MODE
    assert call(lib, kind, mode=mcl.MC_SSC, topk=-1) == mcl.MC_ERR_TOPK
    assert call(lib, kind, mode=mcl.MC_SSC, topk=65, L=4096) == mcl.MC_ERR_TOPK


TOKEN = ["q", "k", "v", "u", "la", "be"]


def delta_step(lib, **kw):
    a = {n: FAKE for n in TOKEN + ["states", "kbar", "online", "ksum", "y"]} | dict(d=16, seg=16, mode=1, topk=0, t=0, n_max=4) | kw
    return lib.mc_decode_step_delta(*(a[n] for n in TOKEN), 1, 1, a["d"], a["seg"], a["mode"], a["topk"], a["t"], a["states"],
                                    a["kbar"], a["online"], a["ksum"], a["n_max"], a["y"], 1, None)


def evict_step(lib, **kw):
    caches = ["states", "kbar", "mass", "slot_seg", "online", "ksum"]
    a = {n: FAKE for n in TOKEN + caches + ["y"]} | dict(d=16, seg=16, mode=1, topk=0, t=0, protect=1, n_max=4) | kw
    return lib.mc_decode_step_evict(*(a[n] for n in TOKEN), 1, 1, a["d"], a["seg"], a["mode"], a["topk"], a["t"], a["protect"],
                                    *(a[n] for n in caches), a["n_max"], a["y"], 1, None)


def test_decode_arguments(lib):
    for step in (delta_step, evict_step):
        for n in ("q", "k", "v", "u", "states", "kbar", "online", "ksum", "y"):
            assert step(lib, **{n: None}) == mcl.MC_ERR_NULL, n
            assert step(lib, **{n: FAKE + 4}) == mcl.MC_ERR_ALIGN, n
        for bad in (dict(t=-1), dict(d=24), dict(seg=0), dict(n_max=0), dict(n_max=65)):
            assert step(lib, **bad) == mcl.MC_ERR_SHAPE, bad
        assert step(lib, mode=9) == mcl.MC_ERR_MODE
        assert step(lib, mode=mcl.MC_SSC, topk=-1) == mcl.MC_ERR_TOPK
        assert step(lib, la=None) == mcl.MC_ERR_NULL and step(lib, be=None) == mcl.MC_ERR_NULL  # one without the other
    assert delta_step(lib, t=64) == mcl.MC_ERR_SHAPE  # segment 4 needs a fifth slot
    assert delta_step(lib, la=None, be=None) == mcl.MC_ERR_NULL
    assert delta_step(lib, u=None, mode=mcl.MC_MEAN, q=FAKE + 4) == mcl.MC_ERR_ALIGN
    assert evict_step(lib, t=1 << 30, la=None, be=None, q=FAKE + 4) == mcl.MC_ERR_ALIGN  # any position, either memory
    assert evict_step(lib, mass=None) == mcl.MC_ERR_NULL and evict_step(lib, slot_seg=None) == mcl.MC_ERR_NULL
    assert evict_step(lib, protect=-1) == mcl.MC_ERR_SHAPE and evict_step(lib, protect=4) == mcl.MC_ERR_SHAPE
    for mode in (mcl.MC_RESIDUAL, mcl.MC_MEAN):
        assert evict_step(lib, mode=mode) == mcl.MC_ERR_MODE


def test_compact_arguments(lib):
    caches = ["states", "kbar", "mass", "slot_seg", "online", "ksum"]

    def comp(**kw):
        a = {n: FAKE for n in ["k", "u", "all"] + caches} | dict(L=64, d=16, seg=16, mode=1, topk=0, protect=1, n_max=2, out=FAKE) | kw
        return lib.mc_cache_compact(a["k"], a["u"], a["all"], 1, 1, a["L"], a["d"], a["seg"], a["mode"], a["topk"], a["protect"],
                                    *(a[n] for n in caches), a["n_max"], a["out"], 1, None)
    for n in ["k", "u", "all"] + caches:
        assert comp(**{n: None}) == mcl.MC_ERR_NULL, n
        assert comp(**{n: FAKE + 4}) == mcl.MC_ERR_ALIGN, n
    assert comp(out=FAKE + 4) == mcl.MC_ERR_ALIGN
    for bad in (dict(L=0), dict(d=20), dict(seg=0), dict(n_max=0), dict(n_max=65), dict(protect=-1), dict(protect=3), dict(L=16385, seg=1)):
        assert comp(**bad) == mcl.MC_ERR_SHAPE, bad
    for mode in (mcl.MC_RESIDUAL, mcl.MC_MEAN, 9):
        assert comp(mode=mode) == mcl.MC_ERR_MODE
    assert comp(mode=mcl.MC_SSC, topk=-2) == mcl.MC_ERR_TOPK


def test_python_checks(lib):
    z = torch.zeros(1, 1, 4, 16)
    with pytest.raises(ValueError):
        mcl.mc_forward_delta(z, z, z, z, z[..., 0], z[..., 0], 4, mcl.MC_GRM)  # no CUDA tensors
    with pytest.raises(ValueError):
        mcl.mc_backward_delta(z[0], z, z, z, z, z, z, 4, mcl.MC_GRM)
    with pytest.raises(TypeError):
        mcl.mc_decode_step_evict(mcl.DecodeCache(1, 1, 16, 4, 2, device="cpu"), z, z, z, z, mcl.MC_GRM)
    with pytest.raises(ValueError):
        mcl.EvictingCache(1, 1, 16, 4, 2, device="cpu").copy_(mcl.EvictingCache(1, 1, 16, 4, 3, device="cpu"))
    c = mcl.EvictingCache(1, 2, 16, 4, 3, device="cpu")
    assert c.slot_seg.eq(-1).all() and c.mass.shape == (1, 2, 3)
