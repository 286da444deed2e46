"""pa_qk_norm_rope_append rejects invalid arguments on the host, before any
launch (no GPU needed: every pointer is a fake that is never dereferenced)."""
import ctypes

import pytest

import paged_kv_cache_74_gb300 as pa

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load_library()


def call(lib, fp8, **kw):
    a = dict(out=A, q=2 * A, k=A, v=A, qs=1024, ks=256, vs=256, qw=A, kw=A, eps=1e-6, cs=A, mp=64, rot=128,
             il=0, pos=0, kc=A, vc=A, bt=A, mb=4, qsl=A, sl=A, ns=2, n=4, hq=8, hkv=2, d=128, bs=16, nb=32,
             sk=1.0, sv=1.0, sm=0, st=0)
    a.update(kw)
    vp = ctypes.c_void_p
    args = [vp(a["out"]), vp(a["q"]), vp(a["k"]), vp(a["v"]), a["qs"], a["ks"], a["vs"], vp(a["qw"]), vp(a["kw"]),
            a["eps"], vp(a["cs"]), a["mp"], a["rot"], a["il"], vp(a["pos"]), vp(a["kc"]), vp(a["vc"]),
            vp(a["bt"]), a["mb"], vp(a["qsl"]), vp(a["sl"]), a["ns"], a["n"], a["hq"], a["hkv"], a["d"],
            a["bs"], a["nb"]]
    tail = [vp(a["sm"]), vp(a["st"]), vp(0)]
    if fp8:
        return lib.pa_qk_norm_rope_append_fp8(*args, a["sk"], a["sv"], *tail)
    return lib.pa_qk_norm_rope_append(*args, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(out=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(cs=0), 1), (dict(kc=0), 1),
    (dict(vc=0), 1), (dict(bt=0), 1), (dict(qsl=0), 1), (dict(sl=0), 1),
    (dict(q=A + 8), 1), (dict(out=A + 4), 1), (dict(cs=A + 4), 1), (dict(qw=A + 4), 1), (dict(kw=A + 8), 1),
    (dict(pos=A + 2), 1), (dict(sm=A + 4), 1), (dict(st=A + 2), 1), (dict(bt=A + 2), 1), (dict(qsl=A + 1), 1),
    (dict(qs=1016), 1), (dict(ks=252), 1), (dict(vs=260), 1), (dict(qs=1028), 1),
    (dict(out=A, q=A, qs=1032), 1),            # in place needs contiguous token rows
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(ns=-1), 1), (dict(n=-1), 1), (dict(hq=0), 1), (dict(hkv=0), 1), (dict(nb=0), 1), (dict(bs=0), 1),
    (dict(mb=0), 1), (dict(mp=0), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(rot=0), 2), (dict(rot=24), 2), (dict(rot=144), 2),
    (dict(hq=16384), 2),
    (dict(ns=0), 0), (dict(n=0), 0), (dict(n=0, q=0, k=0), 0),   # nothing to do, nothing launched
])
def test_rejects_invalid_arguments(lib, fp8, kw, expect):
    assert call(lib, fp8, **kw) == expect


@pytest.mark.parametrize("kw", [dict(sk=0.0), dict(sv=-1.0), dict(sk=float("nan")), dict(sv=float("inf"))])
def test_fp8_rejects_bad_scales(lib, kw):
    assert call(lib, True, **kw) == 1


def test_wrapper_needs_cuda_tensors():
    import torch
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.qk_norm_rope_append(x, x, x, x, x, x, x, x, x)
