"""pa_commit_planned_tokens rejects invalid arguments on the host, before any launch (no
GPU needed: every pointer is a fake that is never dereferenced)."""
import ctypes

import pytest

import paged_kv_cache_74_gb300 as pa
from test_step_plan_host import at

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load_library()


def commit(lib, **kw):
    a = dict(kc=at(20), vc=at(40), layers=2, bt=at(0), mb=8, ctx=at(1), new=at(2), seq=at(6), acc=at(3), ma=4, al=at(4),
             nl=at(5), ns=4, hkv=2, d=64, bs=16, nb=64, el=2, st=at(12))
    a.update(kw)
    return lib.pa_commit_planned_tokens(vp(a["kc"]), vp(a["vc"]), a["layers"], vp(a["bt"]), a["mb"], vp(a["ctx"]),
                                        vp(a["new"]), vp(a["seq"]), vp(a["acc"]), a["ma"], vp(a["al"]), vp(a["nl"]),
                                        a["ns"], a["hkv"], a["d"], a["bs"], a["nb"], a["el"], vp(a["st"]), vp(0))


@pytest.mark.parametrize("kw,expect", [
    (dict(seq=0), 1), (dict(seq=at(6) + 2), 1), (dict(nl=at(6)), 1), (dict(seq=at(5) + 12), 1), (dict(seq=at(12)), 1),
    (dict(seq=at(20) + 64), 1), (dict(seq=0, ns=0), 0), (dict(layers=0), 0), (dict(seq=at(1), nl=at(1)), 1),
    (dict(kc=0), 1), (dict(acc=0), 1), (dict(ma=0), 1), (dict(el=4), 2), (dict(ns=70000), 2),
])
def test_rejects_invalid_arguments(lib, kw, expect):
    assert commit(lib, **kw) == expect
