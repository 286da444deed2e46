"""pa_tree_attention rejects invalid arguments on the host, before any launch (no
GPU needed: every pointer is a fake that is never dereferenced)."""
import ctypes

import pytest
import torch

import paged_kv_cache_74_gb300 as pa

A = 0x10000
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load_library()


def call(lib, fp8, **kw):
    a = dict(out=A, q=A, kc=A, vc=A, qsl=A, sl=A, ns=2, tq=10, mql=9, msl=64, bt=A, mb=4, masks=A, words=1, hq=8,
             hkv=2, d=128, bs=16, nb=32, scale=0.125, sk=1.0, sv=1.0, ws=A, wsb=1 << 30)
    a.update(kw)
    args = [vp(a["out"]), vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["qsl"]), vp(a["sl"]), a["ns"], a["tq"], a["mql"],
            a["msl"], vp(a["bt"]), a["mb"], vp(a["masks"]), a["words"], a["hq"], a["hkv"], a["d"], a["bs"], a["nb"],
            a["scale"]]
    if fp8:
        return lib.pa_tree_attention_fp8(*args, a["sk"], a["sv"], vp(a["ws"]), a["wsb"], vp(0))
    return lib.pa_tree_attention(*args, vp(a["ws"]), a["wsb"], vp(0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(out=0), 1), (dict(q=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(bt=0), 1), (dict(sl=0), 1),
    (dict(qsl=0), 1), (dict(masks=0), 1), (dict(masks=A + 4), 1), (dict(qsl=A + 2), 1), (dict(q=A + 8), 1),
    (dict(hq=6, hkv=4), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(msl=65), 1),
    (dict(tq=-1), 1), (dict(mql=-1), 1), (dict(mql=65), 1), (dict(words=0), 1), (dict(words=-1), 1),
    (dict(mql=65, msl=128, mb=8), 1),                       # more rows than the masks have bits
    (dict(words=5), 2), (dict(d=96), 2), (dict(bs=8), 2), (dict(hq=34, hkv=2), 2), (dict(ns=70000), 2),
    (dict(ws=0), 3), (dict(wsb=16), 3), (dict(ws=A + 16), 1),
    (dict(ns=0), 0), (dict(tq=0), 0), (dict(mql=0), 0),
])
def test_rejects_invalid_arguments(lib, fp8, kw, expect):
    assert call(lib, fp8, **kw) == expect


@pytest.mark.parametrize("kw", [dict(sk=0.0), dict(sv=-1.0), dict(sk=float("nan")), dict(sv=float("inf"))])
def test_fp8_rejects_bad_scales(lib, kw):
    assert call(lib, True, **kw) == 1


@pytest.mark.parametrize("args", [(-1, 4, 8, 2, 128, 64), (2, -1, 8, 2, 128, 64), (2, 4, 8, 3, 128, 64),
                                  (2, 4, 8, 2, 80, 64), (2, 4, 8, 2, 128, 0), (70000, 4, 8, 2, 128, 64)])
def test_workspace_size_of_invalid_arguments_is_zero(lib, args):
    assert pa.tree_workspace_size(*args) == 0


def test_workspace_grows_with_the_batch_up_to_a_bound(lib):
    sizes = [pa.tree_workspace_size(s, 4 * s, 8, 2, 128, 4096) for s in (1, 2, 8, 64, 4096)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] == sizes[-2]
    assert pa.tree_workspace_size(1, 4, 8, 2, 64, 4096) < sizes[0]


def test_wrapper_needs_cuda_tensors():
    x = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.tree_attention(q, c, c, x, x[:1], x.view(2, 1)[:1], torch.ones(1, dtype=torch.int64), 1, 16, 0.125)
