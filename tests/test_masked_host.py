"""The masked attention calls reject invalid arguments on the host, before any
launch (no GPU needed: every pointer is a fake that is never dereferenced)."""
import ctypes

import pytest

import paged_kv_cache_74_gb300 as pa

A = 0x10000
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load_library()


def decode(lib, fp8, **kw):
    a = dict(out=A, q=A, kc=A, vc=A, bt=A, mb=4, sl=A, ns=2, msl=64, hq=8, hkv=2, d=128, bs=16, nb=32, scale=0.125,
             sk=1.0, sv=1.0, cap=0.0, slopes=0, starts=0, prefix=0, pt=0, ws=A, wsb=1 << 20)
    a.update(kw)
    head = [vp(a["out"]), vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["bt"]), a["mb"], vp(a["sl"]), a["ns"], a["msl"],
            a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"]]
    tail = [a["cap"], vp(a["slopes"]), vp(a["starts"]), vp(a["prefix"]), a["pt"], vp(a["ws"]), a["wsb"], vp(0)]
    if fp8:
        return lib.pa_decode_masked_fp8(*head, a["sk"], a["sv"], *tail)
    return lib.pa_decode_masked(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(out=0), 1), (dict(q=0), 1), (dict(kc=0), 1), (dict(bt=0), 1), (dict(sl=0), 1), (dict(q=A + 8), 1),
    (dict(hq=6, hkv=4), 1), (dict(msl=65), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(cap=-1.0), 1), (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(cap=1e-45), 1),
    (dict(slopes=A + 2), 1), (dict(starts=A + 2), 1), (dict(prefix=A + 1), 1),
    (dict(pt=24), 1), (dict(pt=-16), 1), (dict(ws=A + 16), 1),
    (dict(d=96), 2), (dict(bs=8), 2), (dict(hq=34, hkv=2), 2), (dict(ns=70000), 2),
    (dict(ws=0), 3), (dict(wsb=16), 3), (dict(ns=0), 0),
])
def test_decode_rejects_invalid_arguments(lib, fp8, kw, expect):
    assert decode(lib, fp8, **kw) == expect


@pytest.mark.parametrize("kw", [dict(sk=0.0), dict(sv=-1.0), dict(sk=float("nan")), dict(sv=float("inf"))])
def test_decode_fp8_rejects_bad_scales(lib, kw):
    assert decode(lib, True, **kw) == 1


def prefill(lib, fp8, **kw):
    a = dict(out=A, q=A, kc=A, vc=A, qsl=A, sl=A, ns=2, tq=10, mql=9, msl=64, bt=A, mb=4, hq=8, hkv=2, d=128,
             bs=16, nb=32, scale=0.125, sk=1.0, sv=1.0, cap=0.0, slopes=0, starts=0, prefix=0, ws=A, wsb=1 << 30)
    a.update(kw)
    head = [vp(a["out"]), vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["qsl"]), vp(a["sl"]), a["ns"], a["tq"],
            a["mql"], a["msl"], vp(a["bt"]), a["mb"], a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"]]
    tail = [a["cap"], vp(a["slopes"]), vp(a["starts"]), vp(a["prefix"]), vp(a["ws"]), a["wsb"], vp(0)]
    if fp8:
        return lib.pa_prefill_varlen_masked_fp8(*head, a["sk"], a["sv"], *tail)
    return lib.pa_prefill_varlen_masked(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(out=0), 1), (dict(q=0), 1), (dict(qsl=0), 1), (dict(qsl=A + 2), 1), (dict(sl=0), 1), (dict(mql=65), 1),
    (dict(tq=-1), 1), (dict(scale=0.0), 1), (dict(cap=-1.0), 1), (dict(cap=float("nan")), 1), (dict(cap=1e-45), 1),
    (dict(slopes=A + 2), 1), (dict(starts=A + 2), 1), (dict(prefix=A + 1), 1), (dict(ws=A + 16), 1),
    (dict(d=96), 2), (dict(bs=8), 2), (dict(hq=34, hkv=2), 2),
    (dict(ws=0), 3), (dict(wsb=16), 3), (dict(ns=0), 0), (dict(tq=0), 0),
])
def test_prefill_rejects_invalid_arguments(lib, fp8, kw, expect):
    assert prefill(lib, fp8, **kw) == expect


@pytest.mark.parametrize("kw", [dict(sk=0.0), dict(sv=-1.0), dict(sk=float("nan")), dict(sv=float("inf"))])
def test_prefill_fp8_rejects_bad_scales(lib, kw):
    assert prefill(lib, True, **kw) == 1


@pytest.mark.parametrize("ns,tq,hq,hkv,d", [(1, 1, 4, 2, 64), (64, 575, 32, 8, 128), (300, 40000, 16, 1, 128)])
def test_prefill_workspace_holds_the_plan(lib, ns, tq, hq, hkv, d):
    """A call is refused one byte below the size it needs; the plan takes 60
    bytes for each of up to total_q / 128 + num_seqs query tiles."""
    plain = lib.pa_prefill_workspace_size(ns, tq, hq, hkv, d, 4096)
    size = lib.pa_prefill_masked_workspace_size(ns, tq, hq, hkv, d, 4096)
    assert size >= plain + 56 * (tq // 128 + ns) + 4 * ns
    assert lib.pa_prefill_masked_workspace_size(ns, tq, 6, 4, d, 4096) == 0
    assert lib.pa_prefill_masked_workspace_size(ns, -1, hq, hkv, d, 4096) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_workspaces_smaller_than_the_size_are_refused(lib, fp8):
    """One byte below what the size functions say, for every unit layout (the
    sizes cover them all)."""
    for hq, hkv in ((8, 2), (16, 2), (4, 4), (40, 8)):
        size = lib.pa_decode_workspace_size(2, hq, hkv, 128, 64, 0)
        assert decode(lib, fp8, hq=hq, hkv=hkv, wsb=size - 1) == 3
        size = lib.pa_prefill_masked_workspace_size(2, 10, hq, hkv, 128, 64)
        for mql in (1, 9):
            assert prefill(lib, fp8, hq=hq, hkv=hkv, mql=mql, wsb=size - 1) == 3
