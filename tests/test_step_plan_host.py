"""pa_plan_step, pa_release_blocks and pa_commit_tokens reject invalid arguments on
the host, before any launch (no GPU needed: every pointer is a fake that is
never dereferenced)."""
import ctypes

import pytest
import torch

import paged_kv_cache_74_gb300 as pa

A = 0x10000000
STEP = 0x100000  # fakes far enough apart not to overlap


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load_library()


def at(k):
    return A + k * STEP


vp = ctypes.c_void_p


def plan(lib, **kw):
    a = dict(bt=at(0), mb=8, held=at(1), ctx=at(2), new=at(3), ns=4, free=at(4), cap=64, count=at(5), bs=16, nb=64,
             qsl=at(6), sl=at(7), sm=at(8), pos=at(9), mt=32, par=at(10), masks=at(11), words=1, st=at(12))
    a.update(kw)
    return lib.pa_plan_step(vp(a["bt"]), a["mb"], vp(a["held"]), vp(a["ctx"]), vp(a["new"]), a["ns"], vp(a["free"]),
                            a["cap"], vp(a["count"]), a["bs"], a["nb"], vp(a["qsl"]), vp(a["sl"]), vp(a["sm"]),
                            vp(a["pos"]), a["mt"], vp(a["par"]), vp(a["masks"]), a["words"], vp(a["st"]), vp(0))


@pytest.mark.parametrize("kw,expect", [
    (dict(bt=0), 1), (dict(held=0), 1), (dict(ctx=0), 1), (dict(new=0), 1), (dict(free=0), 1), (dict(count=0), 1),
    (dict(qsl=0), 1), (dict(sl=0), 1), (dict(sm=0), 1), (dict(pos=0), 1),
    (dict(masks=0), 1), (dict(words=0), 1), (dict(words=-1), 1), (dict(words=5), 2), (dict(masks=0, words=0, mt=-1), 1),
    (dict(ns=-1), 1), (dict(ns=65536), 2), (dict(mb=0), 1), (dict(cap=0), 1), (dict(bs=0), 1), (dict(nb=0), 1),
    (dict(mb=1 << 27, bs=64), 2),
    (dict(bt=at(0) + 2), 1), (dict(sm=at(8) + 4), 1), (dict(masks=at(11) + 4), 1), (dict(pos=at(9) + 1), 1),
    (dict(sl=at(2)), 1),                 # lengths in place of the context lengths
    (dict(sl=at(2) + 12), 1),            # ... or one entry of them
    (dict(free=at(5)), 1), (dict(qsl=at(3)), 1), (dict(pos=at(10)), 1), (dict(sm=at(11)), 1), (dict(held=at(2)), 1),
    (dict(st=at(7)), 1),
])
def test_plan_step_rejects_invalid_arguments(lib, kw, expect):
    assert plan(lib, **kw) == expect


def release(lib, **kw):
    a = dict(bt=at(0), mb=8, held=at(1), keep=at(2), ns=4, free=at(4), cap=64, count=at(5), bs=16, nb=64, st=at(12))
    a.update(kw)
    return lib.pa_release_blocks(vp(a["bt"]), a["mb"], vp(a["held"]), vp(a["keep"]), a["ns"], vp(a["free"]), a["cap"],
                                 vp(a["count"]), a["bs"], a["nb"], vp(a["st"]), vp(0))


@pytest.mark.parametrize("kw,expect", [
    (dict(bt=0), 1), (dict(held=0), 1), (dict(keep=0), 1), (dict(free=0), 1), (dict(count=0), 1), (dict(ns=-1), 1),
    (dict(ns=65536), 2), (dict(ns=0), 0), (dict(mb=0), 1), (dict(cap=0), 1), (dict(bs=0), 1), (dict(nb=0), 1),
    (dict(keep=at(2) + 2), 1), (dict(keep=at(1)), 1), (dict(free=at(0)), 1), (dict(count=at(4) + 8), 1),
])
def test_release_blocks_rejects_invalid_arguments(lib, kw, expect):
    assert release(lib, **kw) == expect


def commit(lib, **kw):
    a = dict(kc=at(20), vc=at(40), layers=2, bt=at(0), mb=8, ctx=at(1), new=at(2), acc=at(3), ma=4, al=at(4),
             nl=at(5), ns=4, hkv=2, d=64, bs=16, nb=64, el=2, st=at(12))
    a.update(kw)
    return lib.pa_commit_tokens(vp(a["kc"]), vp(a["vc"]), a["layers"], vp(a["bt"]), a["mb"], vp(a["ctx"]),
                                vp(a["new"]), vp(a["acc"]), a["ma"], vp(a["al"]), vp(a["nl"]), a["ns"], a["hkv"],
                                a["d"], a["bs"], a["nb"], a["el"], vp(a["st"]), vp(0))


@pytest.mark.parametrize("kw,expect", [
    (dict(kc=0), 1), (dict(vc=0), 1), (dict(bt=0), 1), (dict(ctx=0), 1), (dict(new=0), 1), (dict(acc=0), 1),
    (dict(al=0), 1), (dict(kc=at(20) + 8), 1), (dict(acc=at(3) + 2), 1), (dict(ns=-1), 1), (dict(layers=-1), 1),
    (dict(ma=0), 1), (dict(mb=0), 1), (dict(hkv=0), 1), (dict(d=0), 1), (dict(bs=0), 1), (dict(nb=0), 1),
    (dict(el=4), 2), (dict(el=1, hkv=1, d=24), 2), (dict(hkv=1, d=12), 2), (dict(ns=70000), 2),
    (dict(ns=0), 0), (dict(layers=0), 0),
    (dict(nl=at(1)), 1), (dict(nl=at(1) + 4), 1), (dict(vc=at(20)), 1), (dict(vc=at(20) + 16), 1),
    (dict(nl=at(20) + 1024), 1),
])
def test_commit_tokens_rejects_invalid_arguments(lib, kw, expect):
    assert commit(lib, **kw) == expect


def test_wrappers_need_cuda_tensors():
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.plan_step(x.view(2, 2), x, x, x, x, x, 16, 4, x, x, x, x)
    with pytest.raises(ValueError):
        pa.release_blocks(x.view(2, 2), x, x, x, x, 16, 4)
    c = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.commit_tokens(c, c, x.view(2, 2), x, x, x.view(2, 2), x)
